"""Vocabulary operators on the GPU against the float64 oracle, element by element.

Tolerances are bounds that follow from the arithmetic, evaluated in float64:
  u   = 2^-8   unit roundoff of bf16, f = 2^-24 that of fp32
  ez  = (d / 16 + 8) 4 f max_iv sum_k |x_ik w_vk| s    a logit: one fp32 addition for each 16 products of the
        matrix instruction, taken at four roundoffs each (its sums may truncate)
  loss: 2 ez + 64 f + 8 f (|lse| + |z_t|)              two logits, the sums, the logs and last roundings
  p:    relative 2 ez + ln2 / 2048 + 32 f              two logits, the log kept in steps of 2^-10 octaves, exp2
  dz:   |dz| u + |coef| p (relative of p) + |coef| 2^-60 (the log's cut at 64 octaves)
  dX, dW: the dz bound carried through the product, plus (K / 16 + 8) 4 f of the absolute product, plus u (bf16)
        or f (fp32) of the result
  embedding gradient: (count + 2) f of the absolute sum, plus the result's rounding
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


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3],
                           np.broadcast_to(tol, got.shape)[bad][:3])


def inputs(n, v, d, seed, spread=1.3, ignored=0.2):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(v, d, generator=g) * (spread / d ** 0.5)).to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g)
    # targets from unforeseen to certain
    x = torch.randn(n, d, generator=g) + torch.rand(n, 1, generator=g) * (12.0 / spread ** 2) * w[t].float()
    if ignored and n > 1:
        t[torch.rand(n, generator=g) < ignored] = -100
    return x.to(torch.bfloat16), w, t, torch.rand(n, generator=g) + 0.5


def check_ce(x, w, t, got, weights=None, mean=True, logit_scale=1.0, grad_scale=1.0, dw_base=None, bf16=True):
    n, d = x.shape
    v = w.shape[0]
    X, W, T = f64(x), f64(w), t.cpu().numpy()
    a = None if weights is None else f64(weights)
    s = float(np.float32(logit_scale))
    r = ovocab.cross_entropy(X, W, T, a, mean, s, float(np.float32(grad_scale)))
    counted = T >= 0
    X = np.where(counted[:, None], X, 0.0)
    ez = (d / 16 + 8) * 4 * F * s * (float((np.abs(X) @ np.abs(W).T).max()) if n else 0.0)
    zt = r["lse"] - r["loss"]
    tol = 2 * ez + 64 * F + 8 * F * (np.abs(r["lse"]) + np.abs(zt))
    for name in ("loss", "lse"):
        if got.get(name) is not None:
            within(got[name], r[name], np.where(counted, tol, 0.0), name)
    if got.get("total") is not None:
        aa = np.where(counted, 1.0 if a is None else a, 0.0)
        norm = aa.sum() if mean else 1.0
        share = np.abs(aa / norm) if norm else aa * 0
        within(got["total"], np.array([r["total"]]), float((share * tol).sum()) + 8 * F * abs(r["total"]), "total")
    coef = grad_scale * s * (np.where(counted, 1.0 if a is None else a, 0.0))
    if mean:
        coef = coef / np.where(counted, 1.0 if a is None else a, 0.0).sum() if coef.any() else coef * 0
    p = np.abs(r["dz"])
    rows = np.arange(n)[counted]
    p[rows, T[counted]] = np.abs(coef[counted]) - p[rows, T[counted]]
    ep = 2 * ez + np.log(2) / 2048 + 32 * F
    edz = np.abs(r["dz"]) * U * (1 + ep) + p * ep + np.abs(coef)[:, None] * 2.0 ** -60
    edz[rows, T[counted]] += 8 * F * np.abs(coef[counted])
    adz, out = np.abs(r["dz"]), U if bf16 else F
    if got.get("dx") is not None:
        e = edz @ np.abs(W) + (v / 16 + 8) * 4 * F * (adz @ np.abs(W))
        within(got["dx"], r["dx"], e + out * (np.abs(r["dx"]) + e) + 1e-38, "dx")
    if got.get("dw") is not None:
        e = edz.T @ np.abs(X) + (n / 16 + 8) * 4 * F * (adz.T @ np.abs(X))
        want = r["dw"] if dw_base is None else r["dw"] + f64(dw_base)
        within(got["dw"], want, e + out * (np.abs(want) + e) + 4 * F * np.abs(want) + 1e-38, "dw")


def run_ce(ops, x, w, t, grads=True, dtype=torch.bfloat16, **kw):
    n = x.shape[0]
    out = {"loss": torch.full((n,), 7.0, device=DEV), "lse": torch.full((n,), 7.0, device=DEV),
           "total": torch.full((1,), 7.0, device=DEV)}
    if grads:
        out["dx"] = torch.full(x.shape, 7.0, device=DEV, dtype=dtype)
        out["dw"] = torch.full(w.shape, 7.0, device=DEV, dtype=dtype)
    ops.cross_entropy(x, w, t, **out, **kw)
    ops.sync()
    return out


CE_SHAPES = [(1, 1, 8), (1, 2, 1), (1, 300, 64), (2, 128, 16), (5, 129, 33), (31, 1000, 72), (64, 257, 256), (130, 1000, 96),
             (257, 513, 1000), (300, 5003, 136), (513, 130, 40), (70, 777, 1001), (129, 40000, 64), (1100, 600, 264),
             (3000, 65, 24), (24, 400, 80), (25, 400, 80), (128, 1030, 200), (257, 1030, 200),
             (2049, 300, 136), (32, 400, 80), (33, 700, 72), (48, 1030, 1000), (63, 5003, 136), (65, 777, 2056)]


@pytest.mark.parametrize("n, v, d", CE_SHAPES)
def test_cross_entropy_sizes(ops, n, v, d):
    x, w, t, a = (q.to(DEV) for q in inputs(n, v, d, seed=n + v + d))
    check_ce(x, w, t, run_ce(ops, x, w, t))
    check_ce(x, w, t, run_ce(ops, x, w, t, weights=a, mean=False, grad_scale=0.25, logit_scale=0.7),
             weights=a, mean=False, grad_scale=0.25, logit_scale=0.7)
    check_ce(x, w, t, run_ce(ops, x, w, t, grads=False))


def large_reference(x, w, t, a):
    """The oracle's formulas and this file's bounds in float64 on the GPU, for heads too large for the host's."""
    n, d = x.shape
    v = w.shape[0]
    counted = t >= 0
    X, W = x.double() * counted[:, None], w.double()
    z = X @ W.T
    ez = (d / 16 + 8) * 4 * F * float((X.abs() @ W.T.abs()).max())
    lse = torch.logsumexp(z, dim=1)
    rows, at = counted.nonzero().squeeze(1), t[counted]
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - z[rows, at]
    coef = (a.double() if a is not None else torch.ones_like(lse)) * counted
    coef = coef / coef.sum()
    p = torch.softmax(z, dim=1) * coef[:, None]
    del z
    dz = p.clone()
    dz[rows, at] -= coef[rows]
    ep = 2 * ez + np.log(2) / 2048 + 32 * F
    edz = dz.abs() * U * (1 + ep) + p * ep + coef[:, None] * 2.0 ** -60
    edz[rows, at] += 8 * F * coef[rows]
    out = {"loss": (loss, (2 * ez + 64 * F + 16 * F * lse.abs()) * counted)}
    for name, k, A, B in (("dx", v, dz, W), ("dw", n, dz.T, X)):
        E = edz if name == "dx" else edz.T
        want = A @ B
        e = E @ B.abs() + (k / 16 + 8) * 4 * F * (A.abs() @ B.abs())
        out[name] = (want, e + U * (want.abs() + e) + 1e-38)
    return out


def test_large_reference_is_the_oracle():
    x, w, t, a = (q.to(DEV) for q in inputs(40, 300, 64, seed=13))
    got = large_reference(x, w, t, a)
    want = ovocab.cross_entropy(f64(x), f64(w), t.cpu().numpy(), f64(a))
    for k in ("loss", "dx", "dw"):
        assert np.allclose(f64(got[k][0]), want[k], rtol=1e-10, atol=1e-14), k


# Heads from 55 and from 180 million entries on take dX with w as the long operand, up to 128 and 256 rows of d logits.
@pytest.mark.parametrize("n, v, d", [(1, 40000, 1000), (24, 36864, 1000), (25, 40009, 1001), (64, 9000, 4096), (65, 40000, 1000),
                                     (120, 62500, 4008), (129, 62500, 4008), (255, 65000, 4000),
                                     (1, 60000, 1000), (24, 14000, 4096), (32, 55100, 1001), (33, 60000, 1000), (64, 27600, 2000), (65, 46000, 4000)])
def test_cross_entropy_large_heads(ops, n, v, d):
    g = torch.Generator(device=DEV).manual_seed(n)
    w = (torch.randn(v, d, generator=g, device=DEV) * (1.3 / d ** 0.5)).to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    x = (torch.randn(n, d, generator=g, device=DEV) + torch.rand(n, 1, generator=g, device=DEV) * 7 * w[t].float()).to(torch.bfloat16)
    if n > 2:
        t[1::5] = -1
    a = torch.rand(n, generator=g, device=DEV) + 0.5
    got = run_ce(ops, x, w, t, weights=a)
    for k, (want, tol) in large_reference(x, w, t, a).items():
        bad = ~((got[k].double() - want).abs() <= tol)
        assert not bool(bad.any()), (k, int(bad.sum()), bad.nonzero()[:3].tolist())


@pytest.mark.parametrize("n, v, d", [(5, 129, 33), (130, 1000, 96), (300, 5003, 136)])
@pytest.mark.parametrize("what", ["fp32", "add_bf16", "add_fp32", "only_dx", "only_dw"])
def test_cross_entropy_outputs(ops, n, v, d, what):
    x, w, t, a = (q.to(DEV) for q in inputs(n, v, d, seed=1))
    t = t.int()
    dtype = torch.float32 if what in ("fp32", "add_fp32") else torch.bfloat16
    out = {}
    if what != "only_dw":
        out["dx"] = torch.empty(n, d, device=DEV, dtype=dtype)
    base = None
    if what != "only_dx":
        out["dw"] = torch.randn(v, d, device=DEV).mul_(1e-2).to(dtype)
        base = out["dw"].clone() if what.startswith("add") else None
    ops.cross_entropy(x, w, t, weights=a, accumulate_dw=base is not None, **out)
    ops.sync()
    check_ce(x, w, t, out, weights=a, dw_base=base, bf16=dtype == torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("add", [False, True])
def test_cross_entropy_in_passes(cuda_lib, dtype, add):
    # 700 tokens x 5056 x 2 bytes in blocks of at most 1 MiB, i.e. 256 tokens: three passes.
    one = cuda_lib.VocabOps(0)
    one.set_tuning(14, 1)
    x, w, t, a = (q.to(DEV) for q in inputs(700, 5003, 136, seed=2))
    dw = torch.randn(w.shape, device=DEV).mul_(1e-2).to(dtype)
    base = dw.clone() if add else None
    out = {"loss": torch.empty(700, device=DEV), "total": torch.empty(1, device=DEV), "dw": dw,
           "dx": torch.empty(x.shape, device=DEV, dtype=dtype)}
    one.cross_entropy(x, w, t, weights=a, accumulate_dw=add, **out)
    one.sync()
    check_ce(x, w, t, out, weights=a, dw_base=base, bf16=dtype == torch.bfloat16)
    one.close()


@pytest.mark.parametrize("pad", [8, 5])
def test_cross_entropy_strided_rows(ops, pad):
    # Rows of a wider buffer: pitch on 16 bytes (read in place) and not (copied); memory between rows stays.
    n, v, d = 200, 1500, 64
    x, w, t, _ = (q.to(DEV) for q in inputs(n, v, d, seed=3))
    def wide(rows, fill):
        return torch.full((rows, d + pad), fill, device=DEV, dtype=torch.bfloat16)
    bx, bw, bdx, bdw = wide(n, float("nan")), wide(v, float("nan")), wide(n, 3.0), wide(v, 3.0)
    bx[:, :d], bw[:, :d] = x, w
    out = {"dx": bdx[:, :d], "dw": bdw[:, :d], "loss": torch.empty(n, device=DEV)}
    ops.cross_entropy(bx[:, :d], bw[:, :d], t, **out)
    ops.sync()
    check_ce(x, w, t, out)
    assert bool((bdx[:, d:] == 3).all()) and bool((bdw[:, d:] == 3).all())


def test_cross_entropy_rows_that_are_not_counted(ops):
    # NaN and infinity where the target is not counted reach nothing.
    x, w, t, a = (q.to(DEV) for q in inputs(300, 700, 64, seed=4, ignored=0.5))
    y = x.clone()
    off = (t < 0).nonzero().squeeze(1)
    assert off.numel() > 50
    y[off[::2]] = float("nan")
    y[off[1::2]] = float("inf")
    for only in (("dx", "dw"), ("dx",)):
        out = {k: torch.empty(s.shape, device=DEV, dtype=torch.bfloat16) for k, s in (("dx", x), ("dw", w)) if k in only}
        out["loss"], out["lse"], out["total"] = torch.empty(300, device=DEV), torch.empty(300, device=DEV), torch.empty(1, device=DEV)
        ops.cross_entropy(y, w, t, weights=a, **out)
        ops.sync()
        check_ce(x, w, t, out, weights=a)


@pytest.mark.parametrize("n", [3, 40, 70, 300])
def test_cross_entropy_certain_tokens_keep_their_digits(ops, n):
    # Logits that are sums of one product, exact in fp32: w's column k, whose id 10 k stands out by 6 + 3 k (a loss
    # down to 1e-8).  What is left, relative to the loss: the rounding of the scale and of z - m, 45 octaves at most
    # (45 ln 2 F each), of the exponentials (8 F), of the few hundred additions in four chains (64 F in the worst
    # case) and of the last steps (8 F); d logits are then rounded to bf16.
    v, d = 500, 8
    g = torch.Generator(device=DEV).manual_seed(n)
    w = (torch.rand(v, d, generator=g, device=DEV) * 4 - 2).to(torch.bfloat16)
    k = torch.arange(d, device=DEV)
    w[10 * k, k] = (6 + 3 * k).to(torch.bfloat16)
    which = torch.arange(n, device=DEV) % d
    x = torch.nn.functional.one_hot(which, d).to(torch.bfloat16)
    t = 10 * which
    loss, lse = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    dw = torch.empty(v, d, device=DEV)
    ops.cross_entropy(x, w, t, loss=loss, lse=lse, dw=dw, mean=False)
    scores = torch.empty(n, device=DEV)
    ops.cross_entropy(x, w, t, loss=scores)
    ops.sync()
    z = w.double().T[which]
    top = z.gather(1, t[:, None])
    rest = (torch.exp(z - top).scatter(1, t[:, None], 0.0)).sum(1)
    want = torch.log1p(rest)
    tol = (2 * 45 * np.log(2) + 80) * F
    for got in (loss, scores):
        within(f64(got), f64(want), tol * f64(want), "loss")
    share = torch.zeros(d, dtype=torch.float64, device=DEV).index_add_(0, which, rest / (1 + rest))
    within(f64(dw[10 * k, k]), -f64(share), (tol + U + n * F) * f64(share), "dw")


def test_cross_entropy_nothing_counted(ops):
    x, w, t, _ = (q.to(DEV) for q in inputs(40, 300, 64, seed=5))
    out = run_ce(ops, x, w, torch.full_like(t, -1))
    assert all(not bool(q.any()) for q in out.values())
    empty = run_ce(ops, x[:0], w, t[:0])
    assert float(empty["total"]) == 0 and not bool(empty["dw"].any())
    kept = torch.ones_like(w)
    ops.cross_entropy(x[:0], w, t[:0], dw=kept, accumulate_dw=True)
    ops.sync()
    assert bool((kept == 1).all())


@pytest.mark.parametrize("spread", [30.0, 0.0])
def test_cross_entropy_far_and_equal_logits(ops, spread):
    # Logits hundreds apart (whole column blocks lie under the log's cut), and all equal.
    x, w, t, _ = (q.to(DEV) for q in inputs(150, 2000, 128, seed=6, spread=1.3))
    x = (x.float() * spread).to(torch.bfloat16)
    check_ce(x, w, t, run_ce(ops, x, w, t))


def test_cross_entropy_weights_of_either_sign(ops):
    # Advantages as weights: negative, zero; and weights that cancel (the mean is over a zero sum: nothing comes out).
    x, w, t, a = (q.to(DEV) for q in inputs(90, 700, 64, seed=14))
    a = a - 1.0
    a[::4] = 0.0
    check_ce(x, w, t, run_ce(ops, x, w, t, weights=a, mean=False), weights=a, mean=False)
    t = t.clamp(min=0)
    a[1::2] = -a[::2]
    out = run_ce(ops, x, w, t, weights=a)
    assert float(out["total"]) == 0 and not bool(out["dx"].any()) and not bool(out["dw"].any())


@pytest.mark.parametrize("n", [20, 300])
def test_cross_entropy_memory_off_16_bytes(ops, n):
    # Every array one element past a boundary.
    x, w, t, a = (q.to(DEV) for q in inputs(n, 700, 72, seed=15))
    def off(q):
        b = torch.zeros(q.numel() + 1, device=DEV, dtype=q.dtype)
        b[1:] = q.reshape(-1)
        return b[1:].view(q.shape)
    for dtype in (torch.bfloat16, torch.float32):
        out = {"loss": off(torch.zeros(n, device=DEV)), "dx": off(torch.zeros(n, 72, device=DEV, dtype=dtype)),
               "dw": off(torch.zeros(700, 72, device=DEV, dtype=dtype)), "total": off(torch.zeros(1, device=DEV))}
        ops.cross_entropy(off(x), off(w), off(t), weights=off(a), **out)
        ops.sync()
        check_ce(x, w, t, out, weights=a, bf16=dtype == torch.bfloat16)
    ids, table = off(t), off(w)
    rows = ops.embed(ids, table, off(x))
    assert torch.equal(rows, torch.where((t >= 0).unsqueeze(1), w[t.clamp(min=0)], torch.zeros_like(x)))
    grad = off(torch.zeros(700, 72, device=DEV))
    ops.embed_grad(ids, rows, grad)
    ops.sync()
    want, absolute = (ovocab.embed_grad(t.cpu().numpy(), q, 700) for q in (f64(rows), np.abs(f64(rows))))
    within(grad, want, n * F * absolute, "grad")


def test_cross_entropy_scores_in_passes(cuda_lib):
    # 7000 tokens x 40 blocks x 8 bytes in at most 1 MiB: three passes, the total over all of them.
    one = cuda_lib.VocabOps(0)
    one.set_tuning(14, 1)
    x, w, t, a = (q.to(DEV) for q in inputs(7000, 5003, 16, seed=16))
    out = {"loss": torch.empty(7000, device=DEV), "lse": torch.empty(7000, device=DEV), "total": torch.empty(1, device=DEV)}
    one.cross_entropy(x, w, t, weights=a, **out)
    one.sync()
    check_ce(x, w, t, out, weights=a)
    one.close()


def test_cross_entropy_past_32_bit_offsets(ops):
    # A head of 600000 x 4096 values, zero but for its last 1000 rows.
    n, v, d, last = 3, 600_000, 4096, 1000
    g = torch.Generator(device=DEV).manual_seed(17)
    w = torch.zeros(v, d, device=DEV, dtype=torch.bfloat16)
    w[-last:] = torch.randn(last, d, generator=g, device=DEV) * (1.3 / d ** 0.5)
    x = torch.randn(n, d, generator=g, device=DEV).to(torch.bfloat16) * 4
    t = torch.tensor([v - 1, v - last, 0], device=DEV)
    out = {"loss": torch.empty(n, device=DEV), "dx": torch.empty_like(x), "dw": torch.empty_like(w)}
    ops.cross_entropy(x, w, t, **out)
    ops.sync()
    z = x.double() @ w[-last:].double().T
    lse = torch.log(torch.exp(z).sum(1) + (v - last))
    zt = torch.stack([z[0, -1], z[1, 0], torch.zeros((), device=DEV, dtype=torch.float64)])
    assert float((out["loss"].double() - (lse - zt)).abs().max()) < 1e-3
    dz = torch.exp(z - lse[:, None])
    dz[0, -1] -= 1
    dz[1, 0] -= 1
    want = dz @ w[-last:].double() / n
    assert float((out["dx"].double() - want).norm() / want.norm()) < 3 * U
    rest = torch.exp(-lse)[:, None].repeat(1, 2)  # rows 0 and v / 2, where w is zero
    rest[2, 0] -= 1
    for rows, part in ((slice(v - last, v), dz), ([0, v // 2], rest)):
        want = part.T @ x.double() / n
        assert float((out["dw"][rows].double() - want).norm() / want.norm()) < 3 * U


def test_cross_entropy_targets_past_the_vocabulary(ops, cuda_lib):
    x, w, t, _ = (q.to(DEV) for q in inputs(60, 300, 64, seed=7))
    bad = t.clone()
    bad[7], bad[11] = 300, 1 << 40
    out = {"loss": torch.empty(60, device=DEV), "dx": torch.empty_like(x), "dw": torch.empty_like(w)}
    ops.cross_entropy(x, w, bad, **out)
    with pytest.raises(cuda_lib.DmuonError) as e:
        ops.sync()
    assert e.value.status == cuda_lib.capi.DMUON_ERR_INVALID_ARG
    t[7] = t[11] = -1
    check_ce(x, w, t, out)
    ops.sync()  # reported once


def test_cross_entropy_gradient_against_differences(ops):
    # total(x + h) - total(x - h) against the mean gradient at the two points times 2h, for steps that bf16 holds.
    # Bounds: fp32 rounding of the totals (2 * 16 f |total|, about 1e-4 here), the gradients' bf16 roundings
    # (4 u of the absolute sum), the trapezoid rule's third-order rest (|dlogit| < 0.25: under 1 % of the step).
    n, v, d = 64, 500, 64
    x, w, t, _ = (q.to(DEV) for q in inputs(n, v, d, seed=8, ignored=0))
    g = torch.Generator().manual_seed(9)
    for which in ("x", "w"):
        base = x if which == "x" else w
        step = (torch.randn(base.shape, generator=g) * float(base.float().std()) * 0.01).to(DEV)
        lo, hi = (base.float() - step).to(torch.bfloat16), (base.float() + step).to(torch.bfloat16)
        tot, grad = [], []
        for q in (lo, hi):
            out = run_ce(ops, q if which == "x" else x, q if which == "w" else w, t, mean=False)
            tot.append(float(out["total"].double()))
            grad.append(out["dx" if which == "x" else "dw"].double())
        delta = hi.double() - lo.double()
        mean_grad = (grad[0] + grad[1]) / 2
        want = float((mean_grad * delta).sum())
        tol = 32 * F * abs(tot[0]) + 4 * U * float((mean_grad * delta).abs().sum()) + 0.01 * abs(want)
        assert abs((tot[1] - tot[0]) - want) <= tol, (which, tot[1] - tot[0], want, tol)


def test_cross_entropy_same_bits_again_and_on_other_streams(ops):
    x, w, t, a = (q.to(DEV) for q in inputs(600, 3000, 200, seed=10))
    x2, w2, t2, _ = (q.to(DEV) for q in inputs(400, 2000, 104, seed=11))
    first, other = run_ce(ops, x, w, t, weights=a), run_ce(ops, x2, w2, t2)
    # Calls on two streams share the handle's scratch: each waits for the one before.
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got, got2 = [], []
    for _ in range(3):
        for s, args, kw, to, like in ((s1, (x, w, t), {"weights": a}, got, first), (s2, (x2, w2, t2), {}, got2, other)):
            with torch.cuda.stream(s):
                out = {k: torch.empty_like(q) for k, q in like.items()}
            ops.cross_entropy(*args, stream=s, **kw, **out)
            to.append(out)
    torch.cuda.synchronize()
    ops.sync()
    for want, outs in ((first, got), (other, got2)):
        for out in outs:
            assert all(torch.equal(want[k], out[k]) for k in want)


def test_vocab_calls_in_a_graph(cuda_lib):
    ops = cuda_lib.VocabOps(0)
    x, w, t, _ = (q.to(DEV) for q in inputs(200, 1500, 64, seed=12))
    want = run_ce(ops, x, w, t)
    rows = torch.empty(200, 64, device=DEV, dtype=torch.bfloat16)
    table = torch.zeros_like(w)
    ops.embed_grad(t, want["dx"], table)
    want_table = table.clone()
    out = {k: torch.zeros_like(q) for k, q in want.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.embed(t, w, rows)
        ops.cross_entropy(x, w, t, **out)
        ops.embed_grad(t, out["dx"], table)
    for _ in range(2):
        table.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[k], out[k]) for k in want) and torch.equal(table, want_table)
    # A larger call outgrows the scratch; the graph's stays.
    big = inputs(1000, 9000, 64, seed=18)
    run_ce(ops, *(q.to(DEV) for q in big[:3]))
    for q in out.values():
        q.zero_()
    table.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want[k], out[k]) for k in want) and torch.equal(table, want_table)
    ops.sync()


# ----------------------------------------------------------------- embedding

def ids_of(kind, n, v, seed):
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(n, generator=g, dtype=torch.float64)
    if kind == "one":
        return torch.full((n,), v - 1)
    if kind == "padding":
        return torch.full((n,), -1)
    if kind == "distinct":
        return torch.randperm(max(n, v), generator=g)[:n] % v
    ids = ((v + 1.0) ** u - 1).long().clamp_(0, v - 1)  # frequent and rare ones
    if kind == "padded":
        ids[torch.rand(n, generator=g) < 0.3] = -100
    return ids


EMBED_SHAPES = [(1, 5, 8, "zipf"), (1, 1, 1, "one"), (17, 300, 768, "padded"), (63, 40, 33, "zipf"), (64, 1, 16, "one"),
                (65, 70000, 24, "distinct"), (300, 50, 2056, "padded"), (4096, 1000, 40, "zipf"), (4097, 600, 64, "padded"),
                (9001, 513, 72, "zipf"), (5000, 7, 16, "one"), (130, 20, 8, "padding"), (20000, 130000, 8, "distinct"),
                (8200, 511, 5, "zipf"), (128, 1, 40, "one"), (128, 33, 776, "padded"), (129, 33, 776, "padded"),
                (100, 90000, 264, "distinct"), (97, 64, 2056, "zipf"), (33, 7, 100, "padding")]
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.float32, torch.bfloat16),
         (torch.bfloat16, torch.float32)]


@pytest.mark.parametrize("n, v, d, kind", EMBED_SHAPES)
@pytest.mark.parametrize("index", [torch.int64, torch.int32])
def test_embed_forward(ops, n, v, d, kind, index):
    ids = ids_of(kind, n, v, seed=n).to(index).to(DEV)
    for table_t, out_t in TYPES:
        table = torch.randn(v, d, device=DEV).to(table_t)
        for scale in (1.0, 27.7):
            out = torch.full((n, d), 7.0, device=DEV, dtype=out_t)
            assert ops.embed(ids, table, out, scale=scale) is out
            ops.sync()
            # one fp32 product and one rounding: the same bits as torch's
            want = table[ids.long().clamp(min=0)].float() * torch.tensor(scale, dtype=torch.float32, device=DEV)
            want = torch.where((ids >= 0).unsqueeze(1), want, torch.zeros_like(want)).to(out_t)
            assert torch.equal(out, want), (table_t, out_t, scale)


@pytest.mark.parametrize("n, v, d, kind", EMBED_SHAPES)
@pytest.mark.parametrize("add", [False, True])
def test_embed_backward(ops, n, v, d, kind, add):
    ids = ids_of(kind, n, v, seed=n + 1).to(DEV)
    host = ids.cpu().numpy()
    counts = np.bincount(host[host >= 0], minlength=v)
    for dout_t, grad_t in TYPES:
        dout = torch.randn(n, d, device=DEV).to(dout_t)
        table = torch.randn(v, d, device=DEV).to(grad_t)
        base = table.clone()
        ops.embed_grad(ids, dout, table, scale=1.5, accumulate=add)
        ops.sync()
        want = ovocab.embed_grad(host, f64(dout), v, 1.5, f64(base) if add else None)
        absolute = ovocab.embed_grad(host, np.abs(f64(dout)), v, 1.5, np.abs(f64(base)) if add else None)
        tol = (counts[:, None] + 3) * F * absolute + (U if grad_t == torch.bfloat16 else F) * np.abs(want) * 1.01
        if add:  # rows that no id names stay as they are
            tol[counts == 0] = 0.0
        within(table, want, tol, (dout_t, grad_t))


@pytest.mark.parametrize("pad", [8, 3])
def test_embed_strided_rows(ops, pad):
    n, v, d = 500, 90, 64
    ids = ids_of("padded", n, v, seed=1).to(DEV)
    table = torch.full((v, d + pad), float("nan"), device=DEV, dtype=torch.bfloat16)
    table[:, :d] = torch.randn(v, d, device=DEV)
    out = torch.full((n, d + pad), 3.0, device=DEV)
    ops.embed(ids, table[:, :d], out[:, :d], scale=0.5)
    grad = torch.full((v, d + pad), 3.0, device=DEV)
    ops.embed_grad(ids, out[:, :d], grad[:, :d])
    ops.sync()
    assert np.array_equal(f64(out[:, :d]), ovocab.embed(ids.cpu().numpy(), f64(table[:, :d]), 0.5))
    want = ovocab.embed_grad(ids.cpu().numpy(), f64(out[:, :d]), v)
    absolute = ovocab.embed_grad(ids.cpu().numpy(), np.abs(f64(out[:, :d])), v)
    within(grad[:, :d], want, n * F * absolute, "grad")
    assert bool((out[:, d:] == 3).all()) and bool((grad[:, d:] == 3).all())


def test_embed_ids_past_the_vocabulary(ops, cuda_lib):
    table = torch.randn(10, 16, device=DEV)
    ids = torch.tensor([0, 10, 9, 1 << 33], device=DEV)
    want = table[torch.tensor([0, 0, 9, 0], device=DEV)] * torch.tensor([[1.0], [0], [1], [0]], device=DEV)
    out = ops.embed(ids, table)
    with pytest.raises(cuda_lib.DmuonError) as e:
        ops.sync()
    assert e.value.status == cuda_lib.capi.DMUON_ERR_INVALID_ARG
    assert torch.equal(out, want)
    grad = torch.full_like(table, 7.0)
    ops.embed_grad(ids, torch.ones(4, 16, device=DEV), grad)
    with pytest.raises(cuda_lib.DmuonError):
        ops.sync()
    ref = torch.zeros_like(table)
    ref[0] = ref[9] = 1
    assert torch.equal(grad, ref)


def test_embed_empty_list(ops):
    table = torch.ones(10, 16, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    assert ops.embed(none, table).shape == (0, 16)
    ops.embed_grad(none, torch.empty(0, 16, device=DEV), table, accumulate=True)
    assert bool((table == 1).all())
    ops.embed_grad(none, torch.empty(0, 16, device=DEV), table)
    ops.sync()
    assert not bool(table.any())


def test_embed_gradient_past_32_bit_offsets(ops):
    # 600000 x 4096 values of a table: row offsets pass 2^31 elements.
    v, d = 600_000, 4096
    table = torch.empty(v, d, device=DEV, dtype=torch.bfloat16)
    table[-1], table[0] = 2.0, 1.0
    ids = torch.tensor([v - 1, 0, v - 1], device=DEV)
    out = ops.embed(ids, table)
    ops.sync()
    assert bool((out[::2] == 2).all()) and bool((out[1] == 1).all())
    ops.embed_grad(ids, out, table)
    ops.sync()
    assert bool((table[-1] == 4).all()) and bool((table[0] == 1).all())
    assert not bool(table[1:-1:1000].any()) and not bool(table[-2].any())


def test_wrapper_checks(ops):
    x = torch.zeros(4, 16, device=DEV, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    for bad in (dict(x=x.float()), dict(w=x[:, :8]), dict(targets=t[:3]), dict(targets=t.float()), dict(x=x.t()),
                dict(dx=torch.zeros(4, 15, device=DEV)), dict(loss=torch.zeros(4, device=DEV, dtype=torch.float64)),
                dict(weights=torch.zeros(8, device=DEV)[::2]), dict(x=torch.zeros(16, device=DEV, dtype=torch.bfloat16))):
        with pytest.raises((TypeError, ValueError)):
            ops.cross_entropy(**{**dict(x=x, w=x, targets=t), **bad})
    with pytest.raises(TypeError):
        ops.embed(t.float(), x)
    with pytest.raises(ValueError):
        ops.embed(t, x, torch.zeros(3, 16, device=DEV))
    with pytest.raises(ValueError):
        ops.embed(t, torch.zeros(1, 16, device=DEV, dtype=torch.bfloat16).expand(4, 16))


@pytest.mark.parametrize("n", [129, 1024, 1025, 2047, 2048, 2049, 4095, 4096, 4097, 8192, 8193, 65536, 65537, 140000])
@pytest.mark.parametrize("v", [300, 70001, 2000032])
def test_embed_backward_long_lists(ops, n, v):
    # Counted places (up to 2048 entries, or 4096 added), both sorts (one launch up to 65536 entries), one to three
    # digits; whole numbers, so sums are exact.
    ids = ids_of("padded", n, v, seed=n).to(DEV)
    dout = torch.randint(-8, 9, (n, 8), device=DEV).float()
    table = torch.full((v, 8), 7.0, device=DEV)
    ops.embed_grad(ids, dout, table)
    ops.sync()
    want = torch.zeros(v, 8, device=DEV, dtype=torch.float64)
    keep = ids >= 0
    want.index_add_(0, ids[keep], dout[keep].double())
    assert torch.equal(table.double(), want)
    ops.embed_grad(ids, dout, table, accumulate=True)
    ops.sync()
    assert torch.equal(table.double(), 2 * want)
    # Fewer ids after many: what the first call named is zero again.
    ops.embed_grad(ids[: n // 4], dout[: n // 4], table)
    ops.sync()
    want.zero_().index_add_(0, ids[: n // 4][keep[: n // 4]], dout[: n // 4][keep[: n // 4]].double())
    assert torch.equal(table.double(), want)


# ------------------------------------------------------------------- example

def _example():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tied_lm.py")
    spec = importlib.util.spec_from_file_location("tied_lm", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_gradients_against_autograd(cuda_lib):
    # The example's whole backward pass against torch's in fp32 on the same bf16 parameters.  Each bf16 tensor on
    # the way (h, x, dx, da, dh) adds one rounding of u = 2^-8: five of them, in norm, stay below 3 u.
    m = _example()
    model = m.TiedLM(vocab=700, dim=64, hidden=96, tokens=500, seed=3)
    g = torch.Generator().manual_seed(4)
    ids, targets = (torch.randint(0, 700, (500,), generator=g).to(DEV) for _ in range(2))
    loss = model.gradients(ids, targets)
    model.sync()
    p = {k: v.float().requires_grad_() for k, v in model.param.items()}
    h = p["table"][ids]
    x = h + torch.relu(h @ p["A"]) @ p["B"]
    want = torch.nn.functional.cross_entropy(x @ p["table"].T, targets)
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) < 1e-2 * want
    for k in p:
        err = float((model.grad[k].double() - p[k].grad.double()).norm() / p[k].grad.double().norm())
        assert err < 3 * U, (k, err)


def test_example_learns(cuda_lib):
    losses = _example().main(steps=60)
    assert losses[0] > 8.0 and losses[-1] < 0.75 * losses[0], losses
