"""Token log probabilities without a GPU: the oracle against closed forms and
differences, and every argument check of the C entry point (all refusals happen
on the host, before CUDA is touched)."""

import numpy as np
import pytest

from oracle import vocab as ovocab


@pytest.fixture(scope="module")
def mos():
    import matrix_optimizer_step_gb300 as m
    from matrix_optimizer_step_gb300 import build

    build.build()
    m.load_library()
    return m


# -------------------------------------------------------------------- oracle

def test_oracle_uniform_distribution():
    r = ovocab.token_logprobs(np.ones((3, 4)), np.zeros((5, 4)), [0, 4, -1], n_top=3, dentropy=np.ones(3))
    assert np.allclose(r["logprobs"], [-np.log(5), -np.log(5), 0]) and np.allclose(r["entropy"], [np.log(5), np.log(5), 0])
    assert r["top_ids"].tolist() == [[0, 1, 2], [0, 1, 2], [-1, -1, -1]]
    # The entropy is at its maximum.
    assert np.allclose(r["dx"], 0) and np.allclose(r["dw"], 0)


def test_oracle_agrees_with_the_cross_entropy():
    r = np.random.default_rng(1)
    x, w, t = r.normal(size=(6, 5)), r.normal(size=(9, 5)), np.array([0, 8, 3, -7, 3, 2])
    ce = ovocab.cross_entropy(x, w, t, mean=False, logit_scale=0.6)
    lp = ovocab.token_logprobs(x, w, t, 0.6, dlogprobs=-np.ones(6))
    for a, b in (("loss", -lp["logprobs"]), ("lse", lp["lse"]), ("dx", lp["dx"]), ("dw", lp["dw"])):
        assert np.allclose(ce[a], b, rtol=1e-12, atol=1e-14), a


def test_oracle_gradient_against_differences():
    r = np.random.default_rng(3)
    x, w = r.normal(size=(6, 5)), r.normal(size=(9, 5))
    t = np.array([0, 8, 3, -7, 3, 2])
    g, h = r.normal(size=6), r.normal(size=6)

    def loss():
        q = ovocab.token_logprobs(x, w, t, 1.7)
        return (g * q["logprobs"] + h * q["entropy"])[t >= 0].sum()

    got = ovocab.token_logprobs(x, w, t, 1.7, 0, g, h, 0.5)
    step = 1e-5
    for name, arr in (("dx", x), ("dw", w)):
        for idx in np.ndindex(arr.shape):
            keep = arr[idx]
            arr[idx] = keep + step
            up = loss()
            arr[idx] = keep - step
            down = loss()
            arr[idx] = keep
            # second-order differences: error O(h^2) = 1e-10 times third derivatives, plus 1e-16 / h rounding
            assert abs(0.5 * (up - down) / (2 * step) - got[name][idx]) < 1e-8, (name, idx)


# ------------------------------------------------------------------ refusals

BASE = 0x10000000  # plausible, never dereferenced: every case here is refused on the host


def lp_args(capi, **kw):
    a = capi.DmuonLogprobs()
    a.n_tokens, a.vocab, a.dim = 4, 100, 16
    a.x, a.w, a.tokens = BASE, BASE + 0x1000, BASE + 0x10000
    a.ld_x = a.ld_w = a.ld_dx = a.ld_dw = 16
    a.logprobs, a.lse, a.entropy = BASE + 0x20000, BASE + 0x21000, BASE + 0x22000
    a.top_ids, a.top_logprobs, a.n_top = BASE + 0x23000, BASE + 0x24000, 5
    a.dlogprobs, a.dentropy = BASE + 0x25000, BASE + 0x26000
    a.dx, a.dw = BASE + 0x30000, BASE + 0x40000
    a.x_dtype = a.w_dtype = a.dx_dtype = a.dw_dtype = capi.DMUON_DTYPE_BF16
    a.token_dtype = a.top_dtype = capi.DMUON_INDEX_I64
    a.logit_scale = a.grad_scale = 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


INV = "ERR_INVALID_ARG"
LP_BAD = [
    ("ERR_SHAPE", dict(n_tokens=-1)), ("ERR_SHAPE", dict(n_tokens=1 << 31)), ("ERR_SHAPE", dict(vocab=0)),
    ("ERR_SHAPE", dict(vocab=(1 << 24) + 1)), ("ERR_SHAPE", dict(dim=0)), ("ERR_SHAPE", dict(ld_x=15)),
    ("ERR_SHAPE", dict(ld_w=15)), ("ERR_SHAPE", dict(ld_dx=15)), ("ERR_SHAPE", dict(ld_dw=15)),
    (INV, dict(x=None)), (INV, dict(w=None)),
    (INV, dict(logprobs=None, lse=None, entropy=None, top_ids=None, top_logprobs=None, n_top=0, dx=None, dw=None)),
    # what needs tokens, coefficients or gradients without them
    (INV, dict(tokens=None)), (INV, dict(tokens=None, logprobs=None)), (INV, dict(dlogprobs=None, dentropy=None)),
    (INV, dict(dx=None, dw=None)),
    (INV, dict(top_ids=None)), (INV, dict(top_ids=None, n_top=0)), (INV, dict(n_top=0)), (INV, dict(n_top=-1)), (INV, dict(n_top=33)),
    (INV, dict(vocab=4)),
    (INV, dict(logit_scale=0.0)), (INV, dict(logit_scale=-1.0)), (INV, dict(logit_scale=float("nan"))),
    (INV, dict(logit_scale=float("inf"))), (INV, dict(grad_scale=float("nan"))), (INV, dict(flags=1)), (INV, dict(flags=4)),
    ("ERR_DTYPE", dict(x_dtype=0)), ("ERR_DTYPE", dict(w_dtype=0)), ("ERR_DTYPE", dict(dx_dtype=2)),
    ("ERR_DTYPE", dict(dw_dtype=-1)), ("ERR_DTYPE", dict(token_dtype=2)), ("ERR_DTYPE", dict(top_dtype=-1)),
    # written memory shared with anything else
    (INV, dict(dx=BASE)), (INV, dict(dw=BASE + 0x1000 + 100)), (INV, dict(logprobs=BASE + 0x21000)),
    (INV, dict(entropy=BASE + 0x25000 + 12)), (INV, dict(top_ids=BASE + 0x24000 - 152)), (INV, dict(top_logprobs=BASE + 0x10000 + 16)),
    (INV, dict(lse=BASE + 0x26000)),
    # not on their elements' boundaries
    (INV, dict(x=BASE + 1)), (INV, dict(tokens=BASE + 0x10004)), (INV, dict(logprobs=BASE + 0x20002)),
    (INV, dict(top_ids=BASE + 0x23004)), (INV, dict(dw=BASE + 0x40002, dw_dtype=0)), (INV, dict(dentropy=BASE + 0x50001)),
]


@pytest.mark.parametrize("status, kw", LP_BAD, ids=lambda v: str(v)[:40])
def test_token_logprobs_refusals(mos, status, kw):
    capi = mos.capi
    ctx = mos.dmuon_context_create(0)
    try:
        with pytest.raises(mos.DmuonError) as e:
            mos.dmuon_token_logprobs(ctx, lp_args(capi, **kw), 0)
        assert e.value.status == getattr(capi, "DMUON_" + status), (kw, e.value)
        assert "token_logprobs" in str(e.value)
    finally:
        mos.dmuon_context_destroy(ctx)


def test_python_refusals(mos):
    import torch

    ops = mos.VocabOps(0)
    with pytest.raises(TypeError):
        ops.token_logprobs(torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(3, 8, dtype=torch.bfloat16))
