"""Gradient norms, clipping and the clipped step on the GPU.

Tolerances.  A thread adds up to 512 squares (of chunks as the sizes here make them) in four chains of fused steps, 128
each, and a block's threads are joined in ten more additions; each step is off by 2^-24 of the running sum at most, and the
rest is added in 64 bits: a sum of squares is within 2 * 130 * 2^-24 of itself, its root within half of that, and the
result is rounded once.  A scaled value is the rounded product of
the factor (its own error: the norm's, and one rounding) and the gradient, 2^-24, then rounded to its type."""

import math

import numpy as np
import pytest
import torch

from oracle import adamw as oadamw
from oracle import grads as ograds

pytestmark = pytest.mark.gpu

DEV = "cuda"
F = 2.0 ** -24
NORM_TOL = 130 * F + F
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops(cuda_lib):
    o = cuda_lib.GradOps(0)
    yield o
    o.close()


def make(sizes, seed=0, types=(BF, F32), scale=1.0, offset=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        b = torch.zeros(n + offset, device=DEV, dtype=types[i % len(types)])
        b[offset:] = torch.randn(n, generator=g, device=DEV) * scale * (i % 3 + 0.5)
        out.append(b[offset:])
    return out


def f64(t):
    return t.detach().double().cpu().numpy()


def check_norms(got, grads):
    norm, norms = got
    total, each = ograds.norms([f64(g) for g in grads])
    assert abs(float(norm) - total) <= NORM_TOL * total + 1e-45, (float(norm), total)
    if norms is not None:
        for i, (a, b) in enumerate(zip(norms.tolist(), each)):
            assert abs(a - b) <= NORM_TOL * b + 1e-45, (i, a, b)
    return total


SETS = [[1], [0], [7], [8, 0, 1], [5003 * 7, 256, 513], [65536, 65537, 131071], [2048] * 40, [1, 2, 3, 4, 5] * 130, [3_000_001, 5],
        [0, 0, 0], [33] * 513, [1 << 18] * 33]


@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_norms(ops, sizes, offset):
    grads = make(sizes, seed=len(sizes), offset=offset)
    norm, norms, coef = torch.full((1,), 7.0, device=DEV), torch.full((len(sizes),), 7.0, device=DEV), torch.full((1,), 7.0, device=DEV)
    ops.norm(ops.register(grads), norm=norm, norms=norms, coef=coef, max_norm=0.5)
    ops.sync()
    total = check_norms((norm, norms), grads)
    want = ograds.factor(total, 0.5)
    assert abs(float(coef) - want) <= (NORM_TOL + F) * want
    again = ops.norm(grads)
    ops.sync()
    assert torch.equal(again, norm)


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-30, 1e-42, 2.0 ** -149, 2.0 ** 64, 2.0 ** -44])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norms_of_large_and_small_values(ops, value, dtype):
    # Squares past the range of fp32: a norm that fits is right, among zeros and among ordinary tensors.
    big = torch.zeros(70_000, device=DEV, dtype=dtype)
    big[5::700] = value  # 100 of them; zero where the type does not reach so low
    value = float(big[5].double())
    alone = ops.norm([big])
    both = torch.empty(2, device=DEV)
    total = ops.norm([big, torch.ones(9, device=DEV)])
    ops.norm([big, torch.ones(9, device=DEV)], norms=both)
    ops.sync()
    one = 10.0 * value
    if one > 3.4028235e38:
        assert math.isinf(float(alone)) and math.isinf(float(total)) and math.isinf(float(both[0]))
    else:
        # 2^-149 is the step of the smallest results.
        assert abs(float(alone) - one) <= NORM_TOL * one + 2.0 ** -149
        assert abs(float(total) - math.hypot(one, 3.0)) <= NORM_TOL * math.hypot(one, 3.0)
    assert abs(float(both[1]) - 3.0) <= NORM_TOL * 3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [1.9921875, 1.1015625, 1.3359375])
@pytest.mark.parametrize("n", [70_000_000, 700_000_000])
def test_norms_keep_the_bound_of_the_longest_chunks(ops, n, value, dtype):
    # A chunk is 128 KB at most: 256 squares of a bf16 chunk a thread, in four chains of 64, then two joins in the thread, five in the
    # warp and three in the block, 74 steps of 2^-24 each: a sum within 5e-6 of itself, a norm within 2.5e-6 and its rounding.
    # Equal values, whose sums are rounded the same way again and again.  The lengths have chunks of just under 128 KB and of all of it.
    if dtype == F32:
        value, n = value + 2.0 ** -12 + 2.0 ** -19, n // 2
    g = torch.full((n,), value, device=DEV, dtype=dtype)
    norm = ops.norm([g])
    ops.sync()
    want = float(g[0].double()) * math.sqrt(n)
    assert 74 * F <= 5e-6 and abs(float(norm) - want) <= (2.5e-6 + F) * want


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_norms_that_are_not_finite(ops, bad):
    grads = make([5000, 300], seed=3)
    grads[0][77] = bad
    norm, coef, norms = torch.empty(1, device=DEV), torch.empty(1, device=DEV), torch.empty(2, device=DEV)
    out = [torch.empty_like(g) for g in grads]
    ops.clip(ops.register(grads, out), 1.0, norm=norm, norms=norms, coef=coef)
    ops.sync()
    assert math.isnan(float(norm)) if math.isnan(bad) else math.isinf(float(norm))
    assert math.isfinite(float(norms[1]))
    if math.isnan(bad):
        assert math.isnan(float(coef)) and all(bool(torch.isnan(o).all()) for o in out)
    else:
        assert float(coef) == 0 and math.isnan(float(out[0][77]))
        out[0][77] = 0
        assert not any(bool(o.any()) for o in out)


@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("out", ["in place", BF, F32])
def test_clip(ops, sizes, offset, out):
    grads = make(sizes, seed=4, offset=offset)
    before = [g.clone() for g in grads]
    outs = None if out == "in place" else make(sizes, seed=5, types=(out,), offset=offset)
    norms, coef = torch.empty(len(sizes), device=DEV), torch.empty(1, device=DEV)
    norm = ops.clip(ops.register(grads, outs), 0.25, norms=norms, coef=coef)
    ops.sync()
    total = check_norms((norm, norms), before)
    want = ograds.factor(total, 0.25)
    assert abs(float(coef) - want) <= (NORM_TOL + F) * want
    for a, b, g in zip(before, outs or grads, grads):
        # The product in fp32 and its rounding are torch's own.
        assert torch.equal(b, (a.float() * coef).to(b.dtype))
        assert outs is None or torch.equal(a, g)


@pytest.mark.parametrize("shift", [1, 2, 5])
def test_clip_between_alignments(ops, shift):
    # What is read and what is written start at different places within 16 bytes.
    for a in (BF, F32):
        for b in (BF, F32):
            grads, outs = make([5000, 9, 70_000], seed=6, types=(a,)), make([5000, 9, 70_000], seed=7, types=(b,), offset=shift)
            coef = torch.empty(1, device=DEV)
            ops.clip(ops.register(grads, outs), 0.25, coef=coef)
            ops.sync()
            assert all(torch.equal(o, (g.float() * coef).to(b)) for g, o in zip(grads, outs))


def test_clip_within_the_norm(ops):
    grads = make([4000, 17], seed=6)
    before = [g.clone() for g in grads]
    out = [torch.empty_like(g, dtype=F32) for g in grads]
    for limit in (1e6, float("inf")):
        ops.clip(grads, limit)
        ops.clip(ops.register(grads, out), limit)
        ops.sync()
        for a, b, c in zip(before, grads, out):
            assert torch.equal(a, b) and torch.equal(a.float(), c)


def test_neighbours_are_left_alone(ops):
    # Views of one buffer, with gaps of one element that stay.
    for dtype in (BF, F32):
        flat = torch.ones(40_000, device=DEV, dtype=dtype)
        ends = [0, 1, 9, 4106, 4107, 30_000, 39_999]
        views = [flat[a:b - 1] if b - a > 1 else flat[a:b] for a, b in zip(ends, ends[1:])]
        inside = torch.zeros(40_000, dtype=torch.bool, device=DEV)
        for a, b in zip(ends, ends[1:]):
            inside[a:max(b - 1, a + 1)] = True
        ops.clip(views, 1.0)
        ops.sync()
        assert bool((flat[~inside] == 1).all()) and bool((flat[inside] < 1).all())


def test_scale(ops):
    grads = make([5000, 77, 0], seed=7)
    before = [g.clone() for g in grads]
    coef = torch.tensor([1.7], device=DEV)
    ops.scale(grads, coef)
    ops.sync()
    for a, b in zip(before, grads):
        assert torch.equal(b, (a.float() * coef).to(b.dtype))


def test_empty_list(ops):
    norm, coef = torch.full((1,), 7.0, device=DEV), torch.full((1,), 7.0, device=DEV)
    ops.clip([], 1.0, norm=norm, coef=coef)
    ops.sync()
    assert float(norm) == 0 and float(coef) == 1


def test_large_tensor(ops):
    # Past 2^31 elements, the last ones counted and scaled.
    n = (1 << 31) + 12345
    g = torch.zeros(n, device=DEV, dtype=BF)
    g[-1], g[0], g[1 << 30] = 3.0, 4.0, 12.0
    norm = ops.clip([g], 1.0)
    ops.sync()
    assert abs(float(norm) - 13.0) <= 13 * NORM_TOL
    assert [float(g[-1]), float(g[0]), float(g[1 << 30])] == [float(torch.tensor(q / 13.0).to(BF)) for q in (3.0, 4.0, 12.0)]


def test_replayed_and_on_another_stream(cuda_lib):
    one = cuda_lib.GradOps(0)
    grads = make([70_000, 513, 5], seed=8)
    outs = [torch.empty_like(g, dtype=BF) for g in grads]
    lst = one.register(grads, outs)
    norm, eager = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    one.clip(lst, 1.0, norm=eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        one.clip(lst, 1.0, norm=norm, stream=side)
    torch.cuda.synchronize()
    one.norm(make([2_000_000] * 40, seed=9))  # outgrows the scratch that the graph holds
    for seed in (8, 10):
        for g, new in zip(grads, make([70_000, 513, 5], seed=seed)):
            g.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for o in outs]
        one.clip(lst, 1.0, norm=eager)
        one.sync()
        assert torch.equal(norm, eager) and all(torch.equal(a, b) for a, b in zip(replayed, outs))
    # Calls on two streams share the scratch: each waits for the one before.
    results = [torch.empty(1, device=DEV) for _ in range(20)]
    torch.cuda.synchronize()
    for i, r in enumerate(results):
        one.norm(grads, norm=r, stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(r, eager) for r in results)
    one.close()


# ------------------------------------------------------------ the clipped step

MATS, VECS = [(256, 512), (384, 128), (3, 64, 96), (24, 320)], [4096, 77, 5000]


def owner(mos, grads, v_grads, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = {"W": [torch.randn(s, generator=g, device=DEV) * 0.02 for s in MATS], "vW": [torch.randn(n, generator=g, device=DEV) for n in VECS]}
    st["B"] = [torch.zeros_like(q) for q in st["W"]]
    st["P"] = [torch.empty_like(q, dtype=BF) for q in st["W"]]
    st["m"], st["v"] = [torch.zeros_like(q) for q in st["vW"]], [torch.zeros_like(q) for q in st["vW"]]
    st["vP"] = [torch.empty_like(q, dtype=BF) for q in st["vW"]]
    step = mos.OwnerStep(0)
    step.set_muon(st["W"], st["B"], grads, st["P"])
    step.set_adamw(st["vW"], st["m"], st["v"], v_grads, st["vP"])
    return step, st


MUON = dict(lr=0.02, momentum=0.95, wd=0.01)
ADAMW = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.01, step=3)


@pytest.mark.parametrize("groups", [1, 3])
def test_clipped_step_is_the_step_on_clipped_gradients(cuda_lib, groups):
    # fp32 gradients: the factor times a gradient is the fp32 product wherever it is formed, so the bits are equal.
    g = torch.Generator(device=DEV).manual_seed(2)
    grads = [torch.randn(s, generator=g, device=DEV) for s in MATS]
    v_grads = [torch.randn(n, generator=g, device=DEV) for n in VECS]
    norm, coef = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    step, st = owner(cuda_lib, grads, v_grads)
    if groups > 1:
        step.set_tuning(9, groups)
        step.set_tuning(10, 1)
    keep = [q.clone() for q in grads + v_grads]
    step.step(MUON, ADAMW, max_norm=0.5, norm=norm)
    step.grad_norm(max_norm=0.5, coef=coef)
    step.sync()
    total = check_norms((norm, None), grads + v_grads)
    assert abs(float(coef) - 0.5 / total) <= (NORM_TOL + 2 * F) * 0.5 / total
    assert all(torch.equal(a, b) for a, b in zip(keep, grads + v_grads))
    other, want = owner(cuda_lib, [q * coef for q in grads], [q * coef for q in v_grads])
    other.step(MUON, ADAMW)
    other.sync()
    for k in st:
        for i, (a, b) in enumerate(zip(st[k], want[k])):
            assert torch.equal(a, b), (k, i)
    step.close()
    other.close()


def test_a_factor_of_one_changes_nothing(cuda_lib):
    g = torch.Generator(device=DEV).manual_seed(3)
    grads = [torch.randn(s, generator=g, device=DEV).to(BF) for s in MATS]
    v_grads = [torch.randn(n, generator=g, device=DEV).to(BF) for n in VECS]
    a, sa = owner(cuda_lib, grads, v_grads)
    b, sb = owner(cuda_lib, grads, v_grads)
    a.step(MUON, ADAMW)
    b.step(MUON, ADAMW, max_norm=1e9)
    a.sync()
    b.sync()
    for k in sa:
        assert all(torch.equal(p, q) for p, q in zip(sa[k], sb[k])), k
    a.close()
    b.close()


def test_clipped_adamw_against_the_oracle(cuda_lib):
    # bf16 gradients, the AdamW route alone.  m takes two roundings and the factor's error, v twice the factor's, the step
    # a handful; W moves by lr, so its own rounding dominates: 16 F of what each formula adds up.
    v_grads = make(VECS, seed=4, types=(BF,))
    step, st = owner(cuda_lib, [torch.ones(s, device=DEV, dtype=BF) for s in MATS], v_grads)
    W0 = [f64(q) for q in st["vW"]]
    norm = torch.empty(1, device=DEV)
    step.step(None, ADAMW, max_norm=0.5, norm=norm)
    step.sync()
    total = check_norms((norm, None), v_grads)
    c = 0.5 / (total + 1e-6)
    for i in range(len(VECS)):
        hp = [float(np.float32(ADAMW[k])) for k in ("lr", "beta1", "beta2", "eps", "wd")]
        r = oadamw.adamw_step(W0[i], np.zeros(VECS[i]), np.zeros(VECS[i]), c * f64(v_grads[i]), *hp, 3)
        for got, want, rel in ((st["m"][i], r["m"], NORM_TOL + 8 * F), (st["v"][i], r["v"], 2 * NORM_TOL + 8 * F)):
            assert bool((np.abs(f64(got) - want) <= rel * np.abs(want)).all())
        moved = np.abs(r["W"] - W0[i])
        assert bool((np.abs(f64(st["vW"][i]) - r["W"]) <= 4 * F * np.abs(r["W"]) + (2 * NORM_TOL + 32 * F) * moved + 1e-9 * hp[0]).all())
    step.close()


def test_clipped_step_replayed(cuda_lib):
    g = torch.Generator(device=DEV).manual_seed(5)
    grads = [torch.randn(s, generator=g, device=DEV).to(BF) for s in MATS]
    v_grads = [torch.randn(n, generator=g, device=DEV).to(BF) for n in VECS]
    a, sa = owner(cuda_lib, grads, v_grads)
    b, sb = owner(cuda_lib, grads, v_grads)
    for s in (a, b):
        s.step(MUON, ADAMW, max_norm=0.5)
        s.step(MUON, ADAMW, max_norm=0.5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.step(MUON, ADAMW, stream=side, max_norm=0.5)
    torch.cuda.synchronize()
    for seed in (6, 7):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for q in grads + v_grads:
            q.copy_(torch.randn(q.shape, generator=g, device=DEV) * seed)
        torch.cuda.synchronize()
        a.step(MUON, ADAMW, max_norm=0.5)
        graph.replay()
        torch.cuda.synchronize()
    for k in sa:
        assert all(torch.equal(p, q) for p, q in zip(sa[k], sb[k])), k
    a.close()
    b.close()


def test_clipped_steps_of_two_routes_on_two_streams(cuda_lib):
    # Each route's step behind a long wait on its own stream, with norms far apart, against the same steps in order.
    g = torch.Generator(device=DEV).manual_seed(11)
    grads = [torch.randn(s, generator=g, device=DEV) for s in MATS]
    v_grads = [torch.randn(n, generator=g, device=DEV) * 1e3 for n in VECS]
    a, sa = owner(cuda_lib, grads, v_grads)
    b, sb = owner(cuda_lib, grads, v_grads)
    norms = [torch.empty(1, device=DEV) for _ in range(4)]
    b.step(MUON, None, max_norm=0.5, norm=norms[2])
    b.sync()
    b.step(None, ADAMW, max_norm=0.5, norm=norms[3])
    b.sync()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(one):
        torch.cuda._sleep(20_000_000)
    a.step(MUON, None, stream=one, max_norm=0.5, norm=norms[0])
    a.step(None, ADAMW, stream=two, max_norm=0.5, norm=norms[1])
    torch.cuda.synchronize()
    assert torch.equal(norms[0], norms[2]) and torch.equal(norms[1], norms[3])
    for k in sa:
        assert all(torch.equal(p, q) for p, q in zip(sa[k], sb[k])), k
    a.close()
    b.close()


def test_policy_step(cuda_lib):
    # The operators together, as a policy-gradient step uses them: scores, a loss in torch, gradients, the clipped step.
    ops = cuda_lib.VocabOps(0)
    g = torch.Generator(device=DEV).manual_seed(6)
    n, v, d = 200, 1000, 64
    head = torch.randn(v, d, generator=g, device=DEV) * 0.1
    param = head.to(BF)
    W = param.double().requires_grad_()
    state = [torch.zeros_like(head) for _ in range(2)]
    grad = torch.empty(v, d, device=DEV, dtype=BF)
    step = cuda_lib.OwnerStep(0)
    step.set_adamw([head], [state[0]], [state[1]], [grad], [param])
    x = torch.randn(n, d, generator=g, device=DEV).to(BF)
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    advantage = torch.randn(n, generator=g, device=DEV)
    dx, norm = torch.empty_like(x), torch.empty(1, device=DEV)
    lp, ent = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    ids, tops = torch.empty(n, 5, device=DEV, dtype=torch.int64), torch.empty(n, 5, device=DEV)
    ops.token_logprobs(x, param, t, logprobs=lp, entropy=ent, top_ids=ids, top_logprobs=tops)
    # Clipped policy ratio against what the sampler saw, with an entropy bonus: torch's own derivative.
    old = lp.clone() + 0.1
    lp_, ent_ = lp.clone().requires_grad_(), ent.clone().requires_grad_()
    ratio = torch.exp(lp_ - old)
    loss = -torch.minimum(ratio * advantage, ratio.clamp(0.8, 1.2) * advantage).mean() - 0.01 * ent_.mean()
    loss.backward()
    ops.token_logprobs(x, param, t, dlogprobs=lp_.grad, dentropy=ent_.grad, dx=dx, dw=grad)
    before = head.clone()
    step.step(None, dict(ADAMW, step=1), max_norm=1e-3, norm=norm)
    ops.sync()
    step.sync()
    # Autograd of the same loss in 64 bits.
    X = x.double().requires_grad_()
    logp = torch.log_softmax(X @ W.T, dim=1)
    LP, H = logp[torch.arange(n, device=DEV), t], -(logp.exp() * logp).sum(1)
    R = torch.exp(LP - old.double())
    (-torch.minimum(R * advantage.double(), R.clamp(0.8, 1.2) * advantage.double()).mean() - 0.01 * H.mean()).backward()
    # A d logit's rounding and a result's to bf16, half a step of 2^-8 each at most, and 2^-11 for the step of its log.
    for got, want in ((dx, X.grad), (grad, W.grad)):
        assert float((got.double() - want).norm()) <= 3 * 2.0 ** -9 * float(want.norm())
    assert abs(float(norm) - float(grad.double().norm())) <= NORM_TOL * float(norm)
    assert bool((ids[:, 0] == torch.argmax(logp, dim=1)).all())
    r = oadamw.adamw_step(f64(before), np.zeros((v, d)), np.zeros((v, d)), f64(grad) * (1e-3 / (float(norm) + 1e-6)),
                          *(float(np.float32(ADAMW[k])) for k in ("lr", "beta1", "beta2", "eps", "wd")), 1)
    # The first step moves a weight by lr g / (|g| + eps): the gradient's sign, and less where it is next to eps.  Errors as above.
    assert bool((np.abs(f64(head) - r["W"]) <= 4 * F * np.abs(r["W"]) + (2 * NORM_TOL + 64 * F) * 1e-3).all())
    assert torch.equal(param, head.to(BF))
    ops.close()
    step.close()
