"""Token log probabilities on the GPU against 64 bits, element by element.

Tolerances are bounds that follow from the arithmetic, evaluated in float64 (units as in
test_gpu_vocab.py: u = 2^-8, f = 2^-24; bf16 and fp32 round by half a step, 2^-9 and 2^-25 of a value at
most, and the bounds take a whole one):
  ez  = (d / 16 + 8) 4 f max_iv sum_k |x_ik w_vk| s + 4 f max|z|   a logit: the matrix instruction's sums, and the scale
  logprob, lse:  2 ez + 64 f + 16 f (|lse| + max |z|)              as the cross entropy's loss
  entropy:  its derivative by z_v is -p_v (ln p_v + H), so D = sum_v p_v |ln p_v + H| carries a logit's error, and the
            sums of positive terms add 64 f of (1 + H); exp2 adds 2^-21 of each term
  top:      ids equal; their log probabilities as logprob
  d logit:  p_v (g + h (ln p_v + H)) with p off by ep = 2 ez + ln2 / 2048 + 32 f of itself, ln p by the same, H by its
            bound; the rounding to bf16, u (two halves: u^2); cut of the logs at 64 octaves
  dX, dW:   the d logits' bound through the product, (K / 16 + 8) 4 f of the absolute product, and the result's rounding
"""

import numpy as np
import pytest
import torch

from oracle import vocab as ovocab

pytestmark = pytest.mark.gpu

U, F = 2.0 ** -8, 2.0 ** -24
DEV = "cuda"


@pytest.fixture(scope="module")
def ops(cuda_lib):
    o = cuda_lib.VocabOps(0)
    yield o
    o.close()


def inputs(n, v, d, seed, ignored=0.2, spread=1.3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (torch.randn(v, d, generator=g, device=DEV) * (spread / d ** 0.5)).to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    x = torch.randn(n, d, generator=g, device=DEV) + torch.rand(n, 1, generator=g, device=DEV) * (12.0 / spread ** 2) * w[t].float()
    if ignored and n > 1:
        t[torch.rand(n, generator=g, device=DEV) < ignored] = -100
    dlp, dent = torch.randn(n, generator=g, device=DEV), torch.randn(n, generator=g, device=DEV) * 0.3
    return x.to(torch.bfloat16), w, t, dlp, dent


def reference(x, w, t, s=1.0, k=0, dlp=None, dent=None, grad_scale=1.0, halves=True, out_u=U):
    """{name: (value, tolerance)} in float64 on the GPU."""
    n, d = x.shape
    v = w.shape[0]
    s, grad_scale = float(np.float32(s)), float(np.float32(grad_scale))
    scored = torch.ones(n, dtype=torch.bool, device=DEV) if t is None else t >= 0
    given = scored & (t is not None)
    X, W = torch.where(scored[:, None], x.double(), 0.0), w.double()
    z = s * (X @ W.T)
    ez = (d / 16 + 8) * 4 * F * s * float((X.abs() @ W.T.abs()).max()) + 4 * F * float(z.abs().max())
    lse = torch.logsumexp(z, dim=1)
    logp = z - lse[:, None]
    p = logp.exp()
    H = -(p * logp.clamp(min=-1e300)).sum(1)
    rows, at = torch.arange(n, device=DEV), (t if t is not None else torch.zeros(n, dtype=torch.int64, device=DEV)).clamp(min=0).long()
    tol = 2 * ez + 64 * F + 16 * F * (lse.abs() + z.abs().amax(1))
    D = (p * (logp + H[:, None]).abs()).sum(1)
    eH = (2 * ez + 2.0 ** -21) * (D + 1) + 64 * F * (1 + H)
    out = {"logprobs": (torch.where(given, logp[rows, at], 0.0), tol * given), "lse": (torch.where(scored, lse, 0.0), tol * scored),
           "entropy": (torch.where(scored, H, 0.0), eH * scored)}
    if k:
        # Which of two logits is larger is decided by sums in 64 bits of the operands alone, laid out the same for all ids.
        exact = torch.cat([(X[i][None, :] * W).sum(1)[None] for i in range(n)]) if n * v * d < 8e9 else z
        ids = torch.sort(exact, dim=1, descending=True, stable=True).indices[:, :k]
        out["top_ids"] = (torch.where(scored[:, None], ids, -1), None)
        out["top_logprobs"] = (torch.where(scored[:, None], logp.gather(1, ids), 0.0), (tol * scored)[:, None].expand(-1, k))
    if dlp is None and dent is None:
        return out
    zero = torch.zeros(n, dtype=torch.float64, device=DEV)
    g = torch.where(given, zero if dlp is None else dlp.double(), 0.0)[:, None]
    h = torch.where(scored, zero if dent is None else dent.double(), 0.0)[:, None]
    dev = logp + H[:, None]
    dz = -p * (g + h * dev)
    dz[rows, at] += g[:, 0]
    ep = 2 * ez + np.log(2) / 2048 + 32 * F
    edz = p * (g + h * dev).abs() * ep + p * h.abs() * (ep + eH[:, None])
    edz[rows, at] += (8 * F + 2 * ez) * (g.abs() + h.abs() * (1 + dev.abs().amax(1, keepdim=True)))[:, 0] * p[rows, at] + 8 * F * g.abs()[:, 0]
    edz += (U * U if halves else U) * (dz.abs() + edz) + (g.abs() + 64 * h.abs()) * 2.0 ** -60
    f = grad_scale * s
    for name, A, E, B, K in (("dx", dz, edz, W, v), ("dw", dz.T, edz.T, X, n)):
        want, e = f * (A @ B), abs(f) * (E @ B.abs() + (K / 16 + 8) * 4 * F * ((A.abs() + E) @ B.abs()))
        out[name] = (want, e + out_u * (want.abs() + e) + 1e-37)
    return out


def check(got, want):
    for name, (value, tol) in want.items():
        if name not in got:
            continue
        a = got[name]
        if tol is None:
            bad = a.long() != value
        else:
            bad = ~((a.double() - value).abs() <= tol)
        assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[:3].tolist(), a[bad][:3].tolist(), value[bad][:3].tolist(),
                                     None if tol is None else tol[bad][:3].tolist())


def outputs(x, w, k, grads=None, ids=torch.int64, types=torch.bfloat16):
    n = x.shape[0]
    out = {c: torch.full((n,), 7.0, device=DEV) for c in ("logprobs", "lse", "entropy")}
    if k:
        out["top_ids"] = torch.full((n, k), 7, device=DEV, dtype=ids)
        out["top_logprobs"] = torch.full((n, k), 7.0, device=DEV)
    if grads:
        out["dx"] = torch.full(x.shape, 7.0, device=DEV, dtype=types)
        out["dw"] = torch.full(w.shape, 7.0, device=DEV, dtype=types)
    return out


SIZES = [(1, 1, 8, 1), (1, 2, 1, 2), (1, 300, 64, 5), (2, 128, 16, 32), (5, 129, 33, 20), (31, 1000, 72, 1), (64, 257, 256, 20),
         (130, 1000, 96, 32), (257, 513, 1000, 20), (300, 5003, 136, 5), (513, 130, 40, 20), (70, 777, 1001, 7), (129, 40000, 64, 20),
         (1100, 600, 264, 3), (3000, 65, 24, 32), (24, 400, 80, 20), (305, 400, 80, 20), (2049, 300, 136, 8), (48, 1030, 1000, 20),
         (65, 777, 2056, 20), (4, 31, 8, 31)]


def test_reference_is_the_oracle():
    x, w, t, dlp, dent = inputs(40, 300, 64, seed=13)
    got = reference(x, w, t, 0.7, 9, dlp, dent, 0.5)
    want = ovocab.token_logprobs(*(q.double().cpu().numpy() for q in (x, w)), t.cpu().numpy(), float(np.float32(0.7)), 9,
                                 dlp.double().cpu().numpy(), dent.double().cpu().numpy(), 0.5)
    for k in got:
        assert np.allclose(got[k][0].cpu().numpy(), want[k], rtol=1e-9, atol=1e-13), k


@pytest.mark.parametrize("n, v, d, k", SIZES)
def test_scores(ops, n, v, d, k):
    x, w, t, _, _ = inputs(n, v, d, seed=n + v + d)
    for s, ids, tokens in ((1.0, torch.int64, t), (1.0 / 0.7, torch.int32, t.int()), (1.0, torch.int64, None)):
        out = outputs(x, w, k, ids=ids)
        if tokens is None:
            del out["logprobs"]
        ops.token_logprobs(x, w, tokens, logit_scale=s, **out)
        ops.sync()
        check(out, reference(x, w, tokens, s, k))
    plain = outputs(x, w, 0)  # without alternatives no log is kept
    ops.token_logprobs(x, w, t, **plain)
    ops.sync()
    check(plain, reference(x, w, t))


@pytest.mark.parametrize("n, v, d, k", SIZES)
def test_gradients(ops, n, v, d, k):
    x, w, t, dlp, dent = inputs(n, v, d, seed=n + v + d + 1)
    for a, b in ((dlp, None), (None, dent), (dlp, dent)):
        out = outputs(x, w, k, grads=True)
        ops.token_logprobs(x, w, t, logit_scale=0.8, dlogprobs=a, dentropy=b, grad_scale=0.25, **out)
        ops.sync()
        check(out, reference(x, w, t, 0.8, k, a, b, 0.25, halves=n <= 128))
    out = outputs(x, w, 0, grads=True)
    del out["logprobs"], out["dx"]
    ops.token_logprobs(x, w, None, dentropy=dent, **out)
    ops.sync()
    check(out, reference(x, w, None, 1.0, 0, None, dent, halves=n <= 128))


@pytest.mark.parametrize("n, v, d", [(5, 129, 33), (300, 5003, 136)])
@pytest.mark.parametrize("what", ["fp32", "fine", "add_bf16", "add_fp32"])
def test_gradient_outputs(ops, n, v, d, what):
    x, w, t, dlp, dent = inputs(n, v, d, seed=2)
    types = torch.bfloat16 if what == "add_bf16" else torch.float32
    out = outputs(x, w, 0, grads=True, types=types)
    base = torch.randn(v, d, device=DEV).mul_(1e-2).to(types)
    out["dw"].copy_(base)
    ops.token_logprobs(x, w, t, dlogprobs=dlp, dentropy=dent, accumulate_dw=what.startswith("add"), fine_grads=what == "fine", **out)
    ops.sync()
    want = reference(x, w, t, 1.0, 0, dlp, dent, halves=n <= 128 or what == "fine", out_u=U if types == torch.bfloat16 else F)
    if what.startswith("add"):
        value, tol = want["dw"]
        want["dw"] = value + base.double(), tol + (U if types == torch.bfloat16 else 4 * F) * (value + base.double()).abs()
    check(out, want)


# Few tokens of a large head: the products with w as the long operand.
@pytest.mark.parametrize("n, v, d", [(1, 60000, 1000), (24, 36864, 1000), (64, 27600, 2000), (65, 46000, 4000), (129, 62500, 1016)])
def test_large_heads(ops, n, v, d):
    x, w, t, dlp, dent = inputs(n, v, d, seed=n)
    out = outputs(x, w, 20, grads=True)
    ops.token_logprobs(x, w, t, dlogprobs=dlp, dentropy=dent, **out)
    ops.sync()
    check(out, reference(x, w, t, 1.0, 20, dlp, dent, halves=n <= 128))


@pytest.mark.parametrize("grads", [False, True])
def test_in_passes(cuda_lib, grads):
    one = cuda_lib.VocabOps(0)
    one.set_tuning(14, 1)  # 256 tokens at a time
    x, w, t, dlp, dent = inputs(700, 5003, 136, seed=3)
    out = outputs(x, w, 20, grads=grads)
    one.token_logprobs(x, w, t, **(dict(dlogprobs=dlp, dentropy=dent) if grads else {}), **out)
    one.sync()
    check(out, reference(x, w, t, 1.0, 20, *((dlp, dent) if grads else ()), halves=False))
    one.close()


@pytest.mark.parametrize("pad", [8, 5])
def test_strided_rows(ops, pad):
    n, v, d = 200, 1500, 64
    x, w, t, dlp, dent = inputs(n, v, d, seed=4)

    def wide(rows, fill):
        return torch.full((rows, d + pad), fill, device=DEV, dtype=torch.bfloat16)

    bx, bw, bdx, bdw = wide(n, float("nan")), wide(v, float("nan")), wide(n, 3.0), wide(v, 3.0)
    bx[:, :d], bw[:, :d] = x, w
    out = outputs(x, w, 20)
    out.update(dx=bdx[:, :d], dw=bdw[:, :d])
    ops.token_logprobs(bx[:, :d], bw[:, :d], t, dlogprobs=dlp, dentropy=dent, **out)
    ops.sync()
    check(out, reference(x, w, t, 1.0, 20, dlp, dent, halves=False))
    assert bool((bdx[:, d:] == 3).all()) and bool((bdw[:, d:] == 3).all())


@pytest.mark.parametrize("n", [20, 300])
def test_memory_off_16_bytes(ops, n):
    x, w, t, dlp, dent = inputs(n, 700, 72, seed=5)

    def off(q):
        b = torch.zeros(q.numel() + 1, device=DEV, dtype=q.dtype)
        b[1:] = q.reshape(-1)
        return b[1:].view(q.shape)

    out = {k: off(q) for k, q in outputs(x, w, 20, grads=True, ids=torch.int32).items()}
    ops.token_logprobs(off(x), off(w), off(t), dlogprobs=off(dlp), dentropy=off(dent), **out)
    ops.sync()
    check(out, reference(x, w, t, 1.0, 20, dlp, dent, halves=n <= 128))


def test_rows_that_are_not_scored(ops):
    # NaN and infinity there reach nothing, and neither do their coefficients.
    x, w, t, dlp, dent = inputs(300, 700, 64, seed=6, ignored=0.5)
    off = (t < 0).nonzero().squeeze(1)
    y, bad = x.clone(), dlp.clone()
    y[off[::2]], y[off[1::2]], bad[off] = float("nan"), float("inf"), float("nan")
    out = outputs(x, w, 20, grads=True)
    ops.token_logprobs(y, w, t, dlogprobs=bad, dentropy=dent, **out)
    ops.sync()
    check(out, reference(x, w, t, 1.0, 20, dlp, dent, halves=False))
    for n in (300, 40):
        none = outputs(x[:n], w, 20, grads=True)
        ops.token_logprobs(y[:n], w, torch.full_like(t[:n], -1), dlogprobs=dlp[:n], **none)
        ops.sync()
        assert bool((none.pop("top_ids") == -1).all())
        assert all(not bool(q.any()) for q in none.values())


def test_rows_without_a_distribution(ops):
    # A NaN in a scored row: NaN and no alternatives there, nothing elsewhere.
    for n in (10, 320):
        x, w, t, _, _ = inputs(n, 700, 64, seed=7, ignored=0)
        y = x.clone()
        y[3, 5] = float("nan")
        out = outputs(x, w, 20)
        ops.token_logprobs(y, w, t, **out)
        ops.sync()
        assert bool((out["top_ids"][3] == -1).all())
        for k in ("logprobs", "lse", "entropy", "top_logprobs"):
            assert bool(torch.isnan(out[k][3]).all()), k
        keep = torch.arange(n, device=DEV) != 3
        want = reference(x, w, t, 1.0, 20)
        check({k: q[keep] for k, q in out.items()}, {k: (a[keep], None if b is None else b[keep]) for k, (a, b) in want.items()})


@pytest.mark.parametrize("n", [5, 310])
def test_equal_logits_go_by_their_ids(ops, n):
    x, w, t, _, _ = inputs(n, 900, 64, seed=8)
    x[1::3] = 0  # every logit 0
    w[400:800:2] = w[399].clone()  # equal rows, more of them than there are candidates at a time
    w[801:] = 0
    out = outputs(x, w, 32)
    ops.token_logprobs(x, w, t, **out)
    ops.sync()
    check(out, reference(x, w, t, 1.0, 32))
    same = w[:1].expand(600, 64).contiguous()  # the whole head one row
    out = outputs(x[:5], same, 32)
    ops.token_logprobs(x[:5], same, torch.zeros(5, dtype=torch.int64, device=DEV), **out)
    ops.sync()
    assert torch.equal(out["top_ids"], torch.arange(32, device=DEV).expand(5, 32))
    assert float((out["entropy"].double() - np.log(600)).abs().max()) <= 1e-5


@pytest.mark.parametrize("n, v", [(6, 40000), (400, 700)])
def test_nearly_equal_logits(ops, n, v):
    # Pairs of entries whose logits differ in the last place of a single small product, far below what 32 bits of the whole
    # logit hold: id 2 i + 1 lies 2^-22 above 2 i, next to a logit of several units.
    d = 64
    x, w, t, _, _ = inputs(n, v, d, seed=9, ignored=0)
    w[1::2] = w[0::2]
    x[:, 0] = 2.0 ** -8
    w[0::2, 0] = 2.0 ** -8
    w[1::2, 0] = 2.0 ** -8 + 2.0 ** -14
    out = outputs(x, w, 20)
    ops.token_logprobs(x, w, t, **out)
    ops.sync()
    assert bool((out["top_ids"][:, 0::2] == out["top_ids"][:, 1::2] + 1).all())
    check(out, reference(x, w, t, 1.0, 20))


@pytest.mark.parametrize("tokens", [True, False])
@pytest.mark.parametrize("n", [4, 40, 600])
def test_logits_that_cancel(ops, n, tokens):
    # Two terms of 300 that cancel but for their rounding, the first and the last of 4096: what the matrix instruction's sums round
    # away is that of a sum of 300 at each step, next to logits of a few units.
    x, w, t, _, _ = inputs(n, 3000, 4096, seed=16)
    x[:, 0] = x[:, 4095] = 17.25
    w[:, 0] = 17.0
    w[:, 4095] = -17.0
    out = outputs(x, w, 20)
    if not tokens:
        del out["logprobs"]
    ops.token_logprobs(x, w, t if tokens else None, **out)
    ops.sync()
    check(out, reference(x, w, t if tokens else None, 1.0, 20))


@pytest.mark.parametrize("tokens", [True, False])
@pytest.mark.parametrize("big", [17.0, 64.0])
@pytest.mark.parametrize("n", [4, 40, 600])
def test_logits_that_cancel_beside_rows_of_zeros(ops, n, big, tokens):
    # As above, but every second row of w alone has the two terms, and the given tokens' rows (without tokens: the first ones)
    # are zeros: what a sum rounds away goes by its own row of w, and no other tells of it.
    x, w, t, _, _ = inputs(n, 3000, 4096, seed=17)
    x[:, 0] = x[:, 4095] = big
    w[:, 0] = w[:, 4095] = 0
    w[1::2, 0] = big
    w[1::2, 4095] = -big
    w[t[t >= 0] if tokens else torch.arange(n, device=DEV)] = 0
    out = outputs(x, w, 20)
    if not tokens:
        del out["logprobs"]
    ops.token_logprobs(x, w, t if tokens else None, **out)
    ops.sync()
    check(out, reference(x, w, t if tokens else None, 1.0, 20))


@pytest.mark.parametrize("n", [6, 300])
def test_infinities_in_the_head(ops, n):
    # Entries shut out by an infinity in their row of w: no probability, and no bound on what else their blocks hold.
    x, w, t, _, _ = inputs(n, 900, 64, seed=18)
    x[:, 7] = x[:, 7].abs() + 1
    out_of = torch.arange(3, 900, 90, device=DEV)
    w[out_of, 7] = float("-inf")
    t[torch.isin(t, out_of)] = -1
    out = outputs(x, w, 32)
    ops.token_logprobs(x, w, t, **out)
    ops.sync()
    keep = torch.ones(900, dtype=torch.bool, device=DEV)
    keep[out_of] = False
    place = keep.nonzero().squeeze(1)
    u = torch.where(t >= 0, (torch.cumsum(keep, 0) - 1)[t.clamp(min=0)], t)
    want = reference(x, w[keep], u, 1.0, 32)
    ids, _ = want["top_ids"]
    want["top_ids"] = (torch.where(ids >= 0, place[ids.clamp(min=0)], ids), None)
    check(out, want)


@pytest.mark.parametrize("spread", [30.0, 0.0])
def test_far_and_equal_logits(ops, spread):
    # Logits hundreds apart: the alternatives lie under the logs' cut.
    for n in (40, 350):
        x, w, t, dlp, dent = inputs(n, 2000, 128, seed=10)
        x = (x.float() * spread).to(torch.bfloat16)
        out = outputs(x, w, 20, grads=True)
        ops.token_logprobs(x, w, t, dlogprobs=dlp, dentropy=dent, **out)
        ops.sync()
        check(out, reference(x, w, t, 1.0, 20, dlp, dent, halves=n <= 128))


@pytest.mark.parametrize("n", [3, 40, 300])
def test_certain_tokens_keep_their_digits(ops, n):
    # As the cross entropy's test of the same name: logits exact in fp32, the log probability down to -1e-8.  The entropy of
    # such a row is r (1 - ln r) with r the rest's share, of terms that are all positive: the logprob's bound, once more for
    # the factor z - z_t (45 octaves, F each) and its sum.
    v, d = 500, 8
    g = torch.Generator(device=DEV).manual_seed(n)
    w = (torch.rand(v, d, generator=g, device=DEV) * 4 - 2).to(torch.bfloat16)
    k = torch.arange(d, device=DEV)
    w[10 * k, k] = (6 + 3 * k).to(torch.bfloat16)
    which = torch.arange(n, device=DEV) % d
    x = torch.nn.functional.one_hot(which, d).to(torch.bfloat16)
    t = 10 * which
    out = outputs(x, w, 1)
    ops.token_logprobs(x, w, t, **out)
    ops.sync()
    z = w.double().T[which]
    far = (z - z.gather(1, t[:, None])).scatter(1, t[:, None], -1e30)
    e = torch.exp(far)
    rest = e.sum(1)
    want = torch.log1p(rest)
    entropy = want - (e * far.clamp(min=-1e3)).sum(1) / (1 + rest)
    tol = (2 * 45 * np.log(2) + 80) * F
    assert bool((out["top_ids"][:, 0] == t).all()) and torch.equal(out["top_logprobs"][:, 0], out["logprobs"])
    assert bool(((out["logprobs"].double() + want).abs() <= tol * want).all())
    assert bool(((out["entropy"].double() - entropy).abs() <= 2 * tol * entropy).all())


@pytest.mark.parametrize("n", [3, 40, 600])
def test_certain_alternatives_without_tokens(ops, n):
    # No token given, logits of 4 to 30 over a sum of 4096 terms, which the matrix instruction's sums cut off towards zero: no
    # probability above 1, falling, and next to 1 off by what the others' share is off by (2 ez of itself, as in `reference`),
    # by the sum's additions and by the rounding of a logit, the product's and its scale's (4 F of it in octaves).
    v, d = 3000, 4096
    g = torch.Generator(device=DEV).manual_seed(19)
    w = (torch.randn(v, d, generator=g, device=DEV) * 0.02).to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    raise_by = torch.linspace(4, 30, n, device=DEV)[:, None]
    x = (torch.randn(n, d, generator=g, device=DEV) * 0.5 + raise_by * w[t].float() / w[t].float().square().sum(1, keepdim=True)).to(torch.bfloat16)
    out = outputs(x, w, 4)
    del out["logprobs"]
    ops.token_logprobs(x, w, None, **out)
    ops.sync()
    check(out, reference(x, w, None, 1.0, 4))
    got = out["top_logprobs"].double()
    assert bool((got <= 0).all()) and bool((got[:, :-1] >= got[:, 1:]).all()) and bool((out["entropy"] >= 0).all())
    z = x.double() @ w.double().T
    top, at = z.max(dim=1)
    rest = torch.exp(z - top[:, None]).scatter(1, at[:, None], 0.0).sum(1)
    ez = (d / 16 + 8) * 4 * F * float((x.double().abs() @ w.double().abs().T).max())
    tol = 2 * ez * rest + 64 * F + 4 * F * top * 1.4427
    sure = rest < 0.9
    assert bool(sure.any()) and bool((((got[:, 0] + torch.log1p(rest)).abs() <= tol) | ~sure).all())


@pytest.mark.parametrize("tokens", [True, False])
@pytest.mark.parametrize("n", [20, 300, 900])
def test_log_probabilities_of_alternatives_fall(ops, n, tokens):
    # A few entries share a row, 0.02 and less apart, and the first two hold terms of 4096 that cancel, for which the matrix
    # instruction's sum loses 0.06: more than lies between them.  With tokens, entries 2 and 3 are next to 0 and 1, closer than the
    # fp32 sum of the given token's logit tells apart.  The values stay in the order of the ids, at 0 or below, and the given
    # token's is its log probability.
    v, d, k, few = 8, 4096, 6, 4 if tokens else 3
    g = torch.Generator(device=DEV).manual_seed(20)
    x = torch.randn(n, d, generator=g, device=DEV)
    w = (torch.randn(1, d, generator=g, device=DEV) * 0.01).expand(v, d).clone()
    x[:, 0] = x[:, d - 1] = 64.0
    w[:, 0] = w[:, d - 1] = 0
    w[:2, 0] = 64.0
    w[:2, d - 1] = -64.0
    x[:, 10] = 8.0
    w[:few, 10] = 4.0
    w[:, 1:4] = 0
    for i in range(few):
        w[i, 1 + (i % 2 if tokens else i)] = 0.02 + (2.0 ** -12 if i >= 2 else 0.0)
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    t = torch.randint(0, few, (n,), generator=g, device=DEV)
    out = outputs(x, w, k)
    if not tokens:
        del out["logprobs"]
    for s in (0.5, 1.0, 2.0):
        ops.token_logprobs(x, w, t if tokens else None, logit_scale=s, **out)
        ops.sync()
        check(out, reference(x, w, t if tokens else None, s, k))
        lp = out["top_logprobs"]
        assert bool((lp <= 0).all()) and bool((lp[:, :-1] >= lp[:, 1:]).all())
        if tokens:
            row, at = (out["top_ids"] == t[:, None]).nonzero(as_tuple=True)
            assert len(row) == n and torch.equal(lp[row, at], out["logprobs"][row])


def test_ids_past_the_vocabulary(cuda_lib):
    one = cuda_lib.VocabOps(0)
    x, w, t, dlp, _ = inputs(50, 300, 64, seed=11)
    t[7] = 300
    out = outputs(x, w, 5, grads=True)
    one.token_logprobs(x, w, t, dlogprobs=dlp, **out)
    with pytest.raises(cuda_lib.DmuonError):
        one.sync()
    t[7] = -1
    check(out, reference(x, w, t, 1.0, 5, dlp, None))
    one.close()


def test_one_call_after_another_and_replayed(cuda_lib):
    # Two sizes on one handle, captured and replayed on new inputs beside eager calls, and on a side stream: the same bits.
    one = cuda_lib.VocabOps(0)
    x, w, t, dlp, dent = inputs(200, 1500, 72, seed=12)
    big = inputs(700, 3000, 72, seed=13)
    eager, replayed = outputs(x, w, 20, grads=True), outputs(x, w, 20, grads=True)

    def call(out, stream=None):
        one.token_logprobs(x, w, t, dlogprobs=dlp, dentropy=dent, stream=stream, **out)

    call(eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(replayed, side)
    torch.cuda.synchronize()
    one.token_logprobs(big[0], big[1], big[2], dlogprobs=big[3], **outputs(big[0], big[1], 5, grads=True))
    for seed in (12, 14):
        for old, new in zip((x, w, t, dlp, dent), inputs(200, 1500, 72, seed=seed)):
            old.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        call(eager)
        one.sync()
        check(eager, reference(x, w, t, 1.0, 20, dlp, dent, halves=False))
        for k in eager:
            assert torch.equal(eager[k], replayed[k]), k
    again = outputs(x, w, 20, grads=True)
    torch.cuda.synchronize()
    call(again, side)
    call(eager)
    torch.cuda.synchronize()
    for k in eager:
        assert torch.equal(eager[k], again[k]), k
    one.close()


def test_nothing_and_defaults(ops):
    x, w, t, dlp, _ = inputs(9, 300, 64, seed=15)
    lp = ops.token_logprobs(x, w, t)
    ops.sync()
    check({"logprobs": lp}, reference(x, w, t))
    empty = outputs(x[:0], w, 3, grads=True)
    ops.token_logprobs(x[:0], w, t[:0], dlogprobs=dlp[:0], **empty)
    ops.sync()
    assert not bool(empty["dw"].any())
