"""Measured cases of what a policy-gradient step needs around the owner's update:

* ``score``   log probabilities of given tokens under a head matrix, with the entropy of each distribution and its
  most likely alternatives (tokens below zero are not scored; ``scale`` is one over the temperature);
* ``policy``  the gradients of hidden states and head from the gradients of those log probabilities and entropies;
* ``norm``    the 2-norm of the gradients of many tensors, together and one by one;
* ``clip``    the same and every gradient times min(1, max_norm / norm), in the type that the step takes;
* ``adamw``   one AdamW step on gradients that are clipped to a global norm on the way.

``own`` false computes them from elementary torch operations in 32 bits, ``own`` true through the package.
"""

import math
import random

import torch

own = False

_handles = {}


def _handle(kind):
    """The one handle of its kind that a user's program keeps for all of its calls."""
    if kind not in _handles:
        import matrix_optimizer_step_gb300 as mos

        _handles[kind] = getattr(mos, kind)(0)
    return _handles[kind]


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_ADAMW = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.01, step=7)


def listed():
    return [
        # One token while generating, with the twenty alternatives that an interface reports at most.
        {"name": "score_1x128256x4096_top20", "op": "score", "tokens": 1, "vocab": 128256, "dim": 4096, "ignored": 0.0,
         "scale": 1.0, "top": 20},
        # A prompt of about a thousand tokens scored against the Llama-3-8B head, a tenth of it not asked for.
        {"name": "score_1000x128256x4096_top5", "op": "score", "tokens": 1000, "vocab": 128256, "dim": 4096, "ignored": 0.1,
         "scale": 1.0, "top": 5},
        # Rollouts of four 1024-token sequences at the GPT-2-small width, sampled at a temperature of 0.7.
        {"name": "score_4096x50257x768_top20", "op": "score", "tokens": 4096, "vocab": 50257, "dim": 768, "ignored": 0.0,
         "scale": 1.0 / 0.7, "top": 20},
        # One batch of 8192 sampled tokens against the Llama-3-8B head, with an entropy bonus.
        {"name": "policy_8192x128256x4096", "op": "policy", "tokens": 8192, "vocab": 128256, "dim": 4096, "ignored": 0.0,
         "scale": 1.0, "bonus": 0.01},
        # Answers only (prompts masked out), every size ragged.
        {"name": "policy_1023x32003x1000", "op": "policy", "tokens": 1023, "vocab": 32003, "dim": 1000, "ignored": 0.4,
         "scale": 1.0 / 0.7, "bonus": 0.01},
        # One short answer: no bonus, the head's gradient is one long write.
        {"name": "policy_24x128256x4096", "op": "policy", "tokens": 24, "vocab": 128256, "dim": 4096, "ignored": 0.0,
         "scale": 1.0, "bonus": 0.0},
        # Every gradient of the Llama-3-8B set: 291 tensors, 8.03e9 elements.
        {"name": "norm_llama3_8b", "op": "norm", "set": "llama3_8b"},
        # A small tied model of three tensors in two types: launch latency.
        {"name": "norm_tied_lm", "op": "norm", "set": "tied_lm"},
        # fp32 accumulators of one Llama-3-8B block, clipped into the bf16 gradients that the step reads.
        {"name": "clip_llama3_8b_block", "op": "clip", "set": "llama3_8b_block", "max_norm": 1.0},
        # Many small matrices and ragged vectors, clipped into one flat buffer (as a collective takes it).
        {"name": "clip_many_small", "op": "clip", "set": "many_small", "max_norm": 1.0},
        # The Llama-3-8B head with its last norm's weight on the AdamW route.
        {"name": "adamw_128256x4096", "op": "adamw", "set": "head", "max_norm": 1.0},
        # What a GPT-2-small model has on the AdamW route: token and position tables and fifty vectors.
        {"name": "adamw_gpt2_small", "op": "adamw", "set": "gpt2_small_adamw", "max_norm": 1.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["score", "score", "policy", "policy", "norm", "clip", "adamw"])
    if op in ("score", "policy"):
        # Widths are multiples of 8 in nearly every model; one in eight here is not.
        dim = _log_int(rng, 256, 4096)
        if rng.random() < 0.875:
            dim = max(256, dim // 8 * 8)
        case = {"op": op, "tokens": _log_int(rng, 1, 8192), "vocab": _log_int(rng, 1000, 128256), "dim": dim,
                "ignored": rng.choice([0.0, 0.0, 0.3]), "scale": rng.choice([1.0, 1.0, 1.0 / 0.7])}
        if op == "score":
            return {**case, "top": rng.choice([0, 1, 5, 20, 20])}
        return {**case, "bonus": rng.choice([0.0, 0.01, 0.01])}
    case = {"op": op, "set": "drawn", "layout": rng.randrange(1 << 30), "tensors": _log_int(rng, 1, 400),
            "elements": _log_int(rng, 1000, 500_000_000 if op == "adamw" else 2_000_000_000)}
    if op != "norm":
        case["max_norm"] = rng.choice([1.0, 1.0, 1e6])
    return case


def _tensors(case):
    """(elements, type of the gradient, type that the step takes) of each tensor of a set."""
    name = case["set"]
    block = [4096 * 4096, 1024 * 4096, 1024 * 4096, 4096 * 4096, 14336 * 4096, 14336 * 4096, 4096 * 14336, 4096, 4096]
    if name == "llama3_8b":
        sizes = [128256 * 4096] + block * 32 + [4096, 128256 * 4096]
        return [(n, "bf16", "bf16") for n in sizes]
    if name == "tied_lm":
        return [(5003 * 256, "f32", "f32"), (256 * 512, "bf16", "bf16"), (512 * 256, "bf16", "bf16")]
    if name == "llama3_8b_block":
        return [(n, "f32", "bf16") for n in block]
    if name == "head":
        return [(128256 * 4096, "bf16", "bf16"), (4096, "bf16", "bf16")]
    if name == "gpt2_small_adamw":
        return [(50257 * 768, "bf16", "bf16"), (1024 * 768, "bf16", "bf16")] + [(768, "bf16", "bf16")] * 50
    if name == "many_small":
        rng = random.Random(17)
        sides = (64, 128, 256, 512, 1024, 2048)
        out = []
        for _ in range(60):
            t = rng.choice(["bf16", "f32"])
            out.append((rng.choice(sides) * rng.choice(sides), t, "bf16"))
            out.append((_log_int(rng, 1, 5000), t, "bf16"))
        return out
    rng = random.Random(case["layout"])
    shares = [math.exp(rng.gauss(0.0, 2.0)) for _ in range(case["tensors"])]
    total = sum(shares)
    types = [("bf16", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")]
    return [(max(1, int(case["elements"] * s / total)), *rng.choice(types)) for s in shares]


def _tokens(n, vocab, g):
    """Ids as text has them: the share of id k falls as 1 / (k + 1)."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return ((vocab + 1.0) ** u - 1.0).long().clamp_(0, vocab - 1)


def _prepare_head(case, s, g):
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    dev = torch.device("cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # Logits of unit-like spread; the given token's is raised by 0 to 12, so that tokens run from unforeseen to certain.
    w = (normal(v, d) * (1.3 / math.sqrt(d))).to(torch.bfloat16)
    t = _tokens(n, v, g)
    x = normal(n, d) + (torch.rand(n, 1, generator=g, device=dev) * (12.0 / 1.69)) * w[t].float()
    if case["ignored"] > 0.0:
        t[torch.rand(n, generator=g, device=dev) < case["ignored"]] = -100
    s.update(x=x.to(torch.bfloat16), w=w, tokens=t)
    if case["op"] == "score":
        k = case["top"]
        s.update(logprobs=torch.empty(n, device=dev), entropy=torch.empty(n, device=dev))
        if k:
            s.update(top_ids=torch.empty(n, k, device=dev, dtype=torch.int64), top_logprobs=torch.empty(n, k, device=dev))
        return s
    # Advantages over the number of tokens, and a bonus for entropy.
    s.update(dlogprobs=normal(n) / n, dentropy=torch.full((n,), -case["bonus"] / n, device=dev) if case["bonus"] else None,
             dx=torch.empty_like(s["x"]), dw=torch.empty_like(w))
    return s


def _flat(sizes, dtype, fill=None):
    """One buffer of the type and a view for each size, at 128-byte steps in it; the gaps hold zeros."""
    step = 128 // dtype.itemsize
    starts, end = [], 0
    for n in sizes:
        starts.append(end)
        end += (n + step - 1) // step * step
    buffer = torch.zeros(end, device="cuda", dtype=dtype)
    views = [buffer[at:at + n] for at, n in zip(starts, sizes)]
    for i, view in enumerate(views):
        for part in view.split(1 << 28) if fill else ():
            part.copy_(fill(i, part.numel()))
    return buffer, views


def _prepare_set(case, s, g):
    sizes = _tensors(case)
    # Magnitudes differ from tensor to tensor, as they do between a model's layers.
    scales = (torch.rand(len(sizes), generator=g, device="cuda") * 4.0 - 6.0).exp_().tolist()

    def normal(i, n):
        return torch.randn(n, generator=g, device="cuda").mul_(scales[i])

    grads = [None] * len(sizes)
    for t, dtype in _TYPES.items():
        of = [i for i, q in enumerate(sizes) if q[1] == t]
        _, views = _flat([sizes[i][0] for i in of], dtype, lambda k, n: normal(of[k], n))
        for i, view in zip(of, views):
            grads[i] = view
    s.update(grads=grads, norm=torch.empty(1, device="cuda"))
    if case["op"] == "norm":
        s["norms"] = torch.empty(len(sizes), device="cuda")
    elif case["op"] == "clip":
        s["outs"], s["flat"] = [None] * len(sizes), {}
        for t, dtype in _TYPES.items():
            of = [i for i, q in enumerate(sizes) if q[2] == t]
            if of:
                s["flat"][t], views = _flat([sizes[i][0] for i in of], dtype)
                for i, view in zip(of, views):
                    s["outs"][i] = view
    else:
        numels = [q[0] for q in sizes]
        s["flat"], f32 = {}, torch.float32
        for name, fill in (("master", lambda i, n: torch.randn(n, generator=g, device="cuda").mul_(0.02)),
                           ("exp_avg", lambda i, n: normal(i, n).mul_(0.5)),
                           ("exp_avg_sq", lambda i, n: normal(i, n).square_())):
            s["flat"][name], s[name] = _flat(numels, f32, fill)
        s["flat"]["param"], s["param"] = _flat(numels, torch.bfloat16, lambda i, n: torch.zeros(n, device="cuda"))
        for w, p in zip(s["master"], s["param"]):
            p.copy_(w)
    if own and case["op"] == "adamw":
        import matrix_optimizer_step_gb300 as mos

        s["owner"] = mos.OwnerStep(0)
        s["owner"].set_adamw(s["master"], s["exp_avg"], s["exp_avg_sq"], grads, s["param"])
    elif own:
        s["list"] = _handle("GradOps").register(grads, s.get("outs"))
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    return _prepare_head(case, s, g) if case["op"] in ("score", "policy") else _prepare_set(case, s, g)


def _plain_top(s, z, lse):
    """The alternatives in falling order.  Which of two close logits is larger is decided in 64 bits, for a few more
    candidates than asked for."""
    k, scale = s["case"]["top"], s["case"]["scale"]
    found = z.topk(min(k + 8, z.shape[1]), dim=1).indices.sort(dim=1).values
    ids, tops = [], []
    for rows in torch.arange(z.shape[0], device=z.device).split(256):
        at = found[rows]
        fine = (s["w"][at].double() * s["x"][rows].double().unsqueeze(1)).sum(dim=2) * scale
        order = fine.sort(dim=1, descending=True, stable=True)
        ids.append(at.gather(1, order.indices[:, :k]))
        tops.append(order.values[:, :k].float() - lse[rows])
    return torch.cat(ids), torch.cat(tops)


def _plain_head(s):
    case = s["case"]
    x, w, t = s["x"].float(), s["w"].float(), s["tokens"]
    given = t >= 0
    at = t.clamp(min=0).unsqueeze(1)
    zero = torch.zeros((), device=x.device)
    z = (x @ w.T) * case["scale"]
    top = z.max(dim=1, keepdim=True).values
    e = (z - top).exp_()
    sums = e.sum(dim=1, keepdim=True)
    log_sums = sums.log()
    # Sum of p ln p, term by term: the entropy with its sign changed.
    plogp = (e * (z - top)).sum(dim=1, keepdim=True) / sums - log_sums
    if case["op"] == "score":
        lse = top + log_sums
        out = {"logprobs": torch.where(given, (z.gather(1, at) - lse).squeeze(1), zero),
               "entropy": torch.where(given, -plogp.squeeze(1), zero)}
        if case["top"]:
            ids, tops = _plain_top(s, z, lse)
            out["top_ids"] = torch.where(given.unsqueeze(1), ids, torch.full_like(ids, -1))
            out["top_logprobs"] = torch.where(given.unsqueeze(1), tops, zero)
        return out
    g = torch.where(given, s["dlogprobs"], zero).unsqueeze(1)
    p = e.div_(sums)
    if s["dentropy"] is None:
        dz = p.mul_(-g)
    else:
        h = torch.where(given, s["dentropy"], zero).unsqueeze(1)
        z.sub_(top).sub_(log_sums).sub_(plogp).mul_(h).add_(g)
        dz = p.mul_(z).neg_()
    dz.scatter_add_(1, at, g)
    dz.mul_(case["scale"])
    return {"dx": (dz @ w).to(s["dx"].dtype), "dw": (dz.T @ x).to(s["dw"].dtype)}


def _plain_norms(s):
    """Norms one by one and together; sums over the tensors in 64 bits."""
    squares = torch.stack([g.float().square().sum() for g in s["grads"]]).double()
    return squares.sqrt().float(), squares.sum().sqrt()


def _plain_set(s):
    case = s["case"]
    norms, norm = _plain_norms(s)
    if case["op"] == "norm":
        return {"norm": norm.float().reshape(1), "norms": norms}
    coef = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    if case["op"] == "clip":
        for g, o in zip(s["grads"], s["outs"]):
            o.copy_(g.float() * coef)
        return {"norm": norm.float().reshape(1), "outs": s["flat"]}
    h = _ADAMW
    step_size, root = h["lr"] / (1.0 - h["beta1"] ** h["step"]), math.sqrt(1.0 - h["beta2"] ** h["step"])
    for g, w, m, v, p in zip(s["grads"], s["master"], s["exp_avg"], s["exp_avg_sq"], s["param"]):
        g = g.float() * coef
        m.mul_(h["beta1"]).add_(g, alpha=1.0 - h["beta1"])
        v.mul_(h["beta2"]).add_(g.square(), alpha=1.0 - h["beta2"])
        w.mul_(1.0 - h["lr"] * h["wd"]).sub_(step_size * (m / (v.sqrt() / root + h["eps"])))
        p.copy_(w)
    return {"norm": norm.float().reshape(1), **s["flat"]}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return _plain_head(s) if op in ("score", "policy") else _plain_set(s)
    if op == "score":
        out = {k: s[k] for k in ("logprobs", "entropy", "top_ids", "top_logprobs") if k in s}
        _handle("VocabOps").token_logprobs(s["x"], s["w"], s["tokens"], logit_scale=case["scale"], **out)
        return out
    if op == "policy":
        _handle("VocabOps").token_logprobs(s["x"], s["w"], s["tokens"], logit_scale=case["scale"], dlogprobs=s["dlogprobs"],
                                    dentropy=s["dentropy"], dx=s["dx"], dw=s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "norm":
        _handle("GradOps").norm(s["list"], norm=s["norm"], norms=s["norms"])
        return {"norm": s["norm"], "norms": s["norms"]}
    if op == "clip":
        _handle("GradOps").clip(s["list"], case["max_norm"], norm=s["norm"])
        return {"norm": s["norm"], "outs": s["flat"]}
    s["owner"].step(None, _ADAMW, max_norm=case["max_norm"], norm=s["norm"])
    return {"norm": s["norm"], **s["flat"]}


def work(case):
    op = case["op"]
    if op in ("score", "policy"):
        n, v, d = case["tokens"], case["vocab"], case["dim"]
        if op == "score":
            # Hidden states, head and tokens read; log probability, entropy and alternatives written.
            return {"bytes": 2 * (n + v) * d + 16 * n + 12 * n * case["top"], "flops": 2 * n * v * d}
        # The same read, with the gradients of both outputs; both gradients written.
        return {"bytes": 4 * (n + v) * d + 16 * n, "flops": 6 * n * v * d}
    sizes = _tensors(case)
    read = sum(n * _SIZE[t] for n, t, _ in sizes)
    n = sum(n for n, _, _ in sizes)
    if op == "norm":
        return {"bytes": read + 4 * len(sizes), "flops": 2 * n}
    if op == "clip":
        return {"bytes": read + sum(n * _SIZE[o] for n, _, o in sizes), "flops": 3 * n}
    # Three states read and written, the parameter written.
    return {"bytes": read + 26 * n, "flops": 16 * n}


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] in ("score", "policy"):
        return _exact_head(case, s)
    squares = torch.zeros(len(s["grads"]), device="cuda", dtype=torch.float64)
    for i, g in enumerate(s["grads"]):
        for part in g.split(1 << 27):
            part = part.double()
            squares[i] += torch.dot(part, part)
    norm = float(squares.sum()) ** 0.5
    total = torch.tensor([norm], device="cuda", dtype=torch.float64)
    if case["op"] == "norm":
        return {"norm": total, "norms": squares.sqrt()}
    factor = min(1.0, case["max_norm"] / (norm + 1e-6))
    sizes = _tensors(case)
    if case["op"] == "clip":
        outs = {}
        for t in s["flat"]:
            outs[t] = _laid_out([factor * g.double() for g, q in zip(s["grads"], sizes) if q[2] == t], 128 // _SIZE[t])
        return {"norm": total, "outs": outs}
    beta1, beta2, t = _ADAMW["beta1"], _ADAMW["beta2"], _ADAMW["step"]
    parts = {"master": [], "exp_avg": [], "exp_avg_sq": []}
    for i, grad in enumerate(s["grads"]):
        grad = factor * grad.double()
        first = beta1 * s["exp_avg"][i].double() + (1.0 - beta1) * grad
        second = beta2 * s["exp_avg_sq"][i].double() + (1.0 - beta2) * grad * grad
        del grad
        move = (first / (1.0 - beta1 ** t)) / (torch.sqrt(second / (1.0 - beta2 ** t)) + _ADAMW["eps"])
        new = s["master"][i].double() - _ADAMW["lr"] * (_ADAMW["wd"] * s["master"][i].double() + move)
        for k, value in zip(parts, (new, first, second)):
            parts[k].append(value)
    out = {k: _laid_out(v, 32) for k, v in parts.items()}
    return {"norm": total, **out, "param": _laid_out(parts["master"], 64)}


def _laid_out(tensors, step):
    """The tensors in one buffer, each at the next multiple of ``step`` elements, zeros between."""
    return torch.cat([torch.nn.functional.pad(t, (0, -t.numel() % step)) for t in tensors])


def _exact_head(case, s):
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    if n * v * d > 2.0e12:
        return None
    score = case["op"] == "score"
    w = s["w"].double()

    def zeros(*shape):
        return torch.zeros(*shape, device="cuda", dtype=torch.float64)

    if score:
        out = {"logprobs": zeros(n), "entropy": zeros(n)}
        if case["top"]:
            out["top_ids"] = torch.full((n, case["top"]), -1, device="cuda", dtype=torch.int64)
            out["top_logprobs"] = zeros(n, case["top"])
    else:
        out = {"dx": zeros(n, d), "dw": zeros(v, d)}
    for block in (s["tokens"] >= 0).nonzero().squeeze(1).split(512):
        x, t = s["x"][block].double(), s["tokens"][block]
        rows = torch.arange(t.numel(), device="cuda")
        logp = torch.log_softmax(torch.mm(x, w.t()) * case["scale"], dim=1)
        p = torch.exp(logp)
        entropy = -(p * logp).sum(dim=1)
        if score:
            out["logprobs"][block] = logp[rows, t]
            out["entropy"][block] = entropy
            if case["top"]:
                # Equal values in the order of their ids.
                values, ids = torch.topk(logp, min(v, case["top"] + 4), dim=1)
                ids, order = torch.sort(ids, dim=1)
                values, order = torch.sort(values.gather(1, order), dim=1, descending=True, stable=True)
                out["top_ids"][block] = ids.gather(1, order)[:, :case["top"]]
                out["top_logprobs"][block] = values[:, :case["top"]]
            continue
        dz = -p * s["dlogprobs"][block].double().unsqueeze(1)
        dz[rows, t] += s["dlogprobs"][block].double()
        if s["dentropy"] is not None:
            dz -= s["dentropy"][block].double().unsqueeze(1) * p * (logp + entropy.unsqueeze(1))
        dz *= case["scale"]
        out["dx"][block] = torch.mm(dz, w)
        out["dw"] += torch.mm(dz.t(), x)
    return out
