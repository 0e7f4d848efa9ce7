"""Cross entropy on the GPU at the sizes of training batches: tiles of both gradient products drawn from one counter,
passes of drawn tiles, lists whose sums have kernels of their own, and every output of large heads.

References and bounds are test_gpu_vocab.py's (float64 on the GPU where the host would take minutes).
"""

import pytest
import torch

from test_gpu_vocab import DEV, F, check_ce, inputs, large_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(cuda_lib):
    o = cuda_lib.VocabOps(0)
    yield o
    o.close()


def batch(n, v, d, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (torch.randn(v, d, generator=g, device=DEV) * (1.3 / d ** 0.5)).to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    x = (torch.randn(n, d, generator=g, device=DEV) + torch.rand(n, 1, generator=g, device=DEV) * 7 * w[t].float()).to(torch.bfloat16)
    t[1::5] = -1
    return x, w, t, torch.rand(n, generator=g, device=DEV) + 0.5


# Both products' tiles are drawn where dW's have 32 k-blocks (2048 tokens) and K is not cut: here dW has 316 tiles of
# 33 blocks, 80 of 36 a pass (two passes), and 790 of 33.  With 2049 x 20000 x 520 W's last column tile is short.
@pytest.mark.parametrize("n, v, d, block_mib", [(2100, 20000, 1000, 0), (4500, 5003, 1000, 24), (2049, 50257, 520, 0)])
@pytest.mark.parametrize("what", ["bf16", "fp32", "add_bf16", "add_fp32"])
def test_drawn_tiles_of_both_gradients(cuda_lib, n, v, d, block_mib, what):
    ops = cuda_lib.VocabOps(0)
    if block_mib:
        ops.set_tuning(14, block_mib)
    x, w, t, a = batch(n, v, d, n)
    dtype = torch.float32 if what.endswith("fp32") else torch.bfloat16
    add = what.startswith("add")
    ref = large_reference(x, w, t, a)
    base = (torch.randn(v, d, device=DEV) * 1e-4).to(dtype)
    for _ in range(2):  # the counters are as before
        out = dict(loss=torch.full((n,), 7.0, device=DEV), dx=torch.full((n, d), 7.0, device=DEV, dtype=dtype), dw=base.clone())
        ops.cross_entropy(x, w, t, weights=a, accumulate_dw=add, **out)
        ops.sync()
        for k, (want, tol) in ref.items():
            if k == "dw" and add:
                want, tol = want + base.double(), tol + (2.0 ** -8 + 8 * F) * (base.double().abs() + want.abs())
            bad = ~((out[k].double() - want).abs() <= tol)
            assert not bool(bad.any()), (k, int(bad.sum()), bad.nonzero()[:3].tolist())
    ops.close()


@pytest.mark.parametrize("n", [16384, 16385, 20001])
@pytest.mark.parametrize("fine", [False, True])
def test_long_lists_with_gradients(ops, n, fine):
    # From 16385 tokens on the factor and the total are sums of whole blocks.
    x, w, t, a = (q.to(DEV) for q in inputs(n, 200, 40, seed=n))
    for mean in (True, False):
        out = dict(loss=torch.empty(n, device=DEV), lse=torch.empty(n, device=DEV), total=torch.empty(1, device=DEV),
                   dx=torch.empty_like(x), dw=torch.empty_like(w))
        ops.cross_entropy(x, w, t, weights=a, mean=mean, fine_grads=fine, **out)
        ops.sync()
        check_ce(x, w, t, out, weights=a, mean=mean)


@pytest.mark.parametrize("n, v, d", [(1, 40000, 1000), (24, 36864, 1000), (64, 27600, 2000), (65, 40000, 1000), (129, 62500, 4008)])
def test_large_heads_log_sums_and_total(ops, n, v, d):
    x, w, t, a = batch(n, v, d, n + 1)
    z = x.double() @ w.double().T
    want = torch.logsumexp(z, 1)
    counted = t >= 0
    loss = (want - z.gather(1, t.clamp(min=0)[:, None])[:, 0]) * counted
    # two logits of d / 16 + 8 additions at four roundoffs each, the sums, logs and last steps (as check_ce)
    ez = (d / 16 + 8) * 4 * F * float((x.double().abs() @ w.double().abs().T).max())
    tol = 2 * ez + 64 * F + 16 * F * want.abs()
    total = float((a.double() * loss).sum() / (a.double() * counted).sum())
    for grads in (False, True):
        out = dict(lse=torch.full((n,), 7.0, device=DEV), total=torch.full((1,), 7.0, device=DEV))
        if grads:
            out.update(dx=torch.empty_like(x), dw=torch.empty_like(w))
        ops.cross_entropy(x, w, t, weights=a, **out)
        ops.sync()
        assert bool(((out["lse"].double() - want * counted).abs() <= tol * counted).all())
        assert abs(float(out["total"]) - total) <= float(tol.max()) + 8 * F * abs(total)


# Few-token logits on both sides of where they leave their own kernel: narrow heads at 48 tokens for scores and at
# 2.2 million logs for gradients (n x v), wide ones at 32.
@pytest.mark.parametrize("n, v, d", [(48, 9000, 512), (49, 9000, 512), (48, 9000, 768), (64, 9000, 768), (15, 140000, 72),
                                     (16, 140000, 72), (32, 68750, 136), (32, 68751, 136), (32, 70000, 2048), (33, 70000, 2048)])
def test_few_tokens_at_the_kernels_borders(ops, n, v, d):
    x, w, t, a = batch(n, v, d, n + d)
    ref = large_reference(x, w, t, a)
    scores, out = torch.empty(n, device=DEV), dict(loss=torch.empty(n, device=DEV), dx=torch.empty_like(x), dw=torch.empty_like(w))
    ops.cross_entropy(x, w, t, weights=a, loss=scores)
    ops.cross_entropy(x, w, t, weights=a, **out)
    ops.sync()
    for k, got in (("loss", scores), *out.items()):
        want, tol = ref[k]
        bad = ~((got.double() - want).abs() <= tol)
        assert not bool(bad.any()), (k, int(bad.sum()), bad.nonzero()[:3].tolist())
