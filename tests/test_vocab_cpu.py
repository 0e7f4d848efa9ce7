"""Vocabulary operators without a GPU: the oracle against closed forms and
differences, and every argument check of the C entry points (all refusals
happen on the host, before CUDA is touched)."""

import ctypes

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

def test_oracle_uniform_logits_closed_form():
    # w = 0: every probability is 1 / v, the loss is log v whatever x is.
    r = ovocab.cross_entropy(np.ones((3, 4)), np.zeros((5, 4)), [0, 4, -1])
    assert np.allclose(r["loss"], [np.log(5), np.log(5), 0], atol=1e-15)
    assert abs(r["total"] - np.log(5)) < 1e-15
    assert np.allclose(r["dx"], 0)
    want = np.full((5, 4), 2 / 5 / 2)
    want[[0, 4]] -= 1 / 2
    assert np.allclose(r["dw"], want)


@pytest.mark.parametrize("mean", [True, False])
def test_oracle_gradient_against_differences(mean):
    r = np.random.default_rng(3)
    x, w = r.normal(size=(6, 5)), r.normal(size=(9, 5))
    t = np.array([0, 8, 3, -7, 3, 2])
    a = r.uniform(0.2, 2.0, 6)
    kw = dict(weights=a, mean=mean, logit_scale=1.7, grad_scale=0.5)
    g = ovocab.cross_entropy(x, w, t, **kw)
    h = 1e-5
    for name, arr in (("dx", x), ("dw", w)):
        for idx in np.ndindex(arr.shape):
            keep = arr[idx]
            arr[idx] = keep + h
            up = ovocab.cross_entropy(x, w, t, **kw)["total"]
            arr[idx] = keep - h
            down = ovocab.cross_entropy(x, w, t, **kw)["total"]
            arr[idx] = keep
            # second-order differences: error O(h^2) = 1e-10 plus 1e-16 / h rounding
            assert abs(0.5 * (up - down) / (2 * h) - g[name][idx]) < 1e-8, (name, idx)


def test_oracle_counts_nothing():
    r = ovocab.cross_entropy(np.full((2, 3), np.nan), np.ones((4, 3)), [-1, -100])
    assert r["total"] == 0 and not r["dx"].any() and not r["dw"].any() and not r["loss"].any()


def test_oracle_embed_is_its_gradients_transpose():
    # <embed(T), G> = <T, embed_grad(G)> for every T and G: the lookup is linear.
    r = np.random.default_rng(4)
    ids = np.array([3, 0, -1, 3, 6, 3])
    T, G = r.normal(size=(7, 5)), r.normal(size=(6, 5))
    assert abs((ovocab.embed(ids, T, 2.5) * G).sum() - (T * ovocab.embed_grad(ids, G, 7, 2.5)).sum()) < 1e-12


# ------------------------------------------------------------------ refusals

def ce_args(capi, **kw):
    a = capi.DmuonCe()
    base = 0x10000000  # plausible, never dereferenced: every case here is refused on the host
    a.n_tokens, a.vocab, a.dim = 4, 100, 16
    a.x, a.w, a.targets = base, base + 0x1000, base + 0x10000
    a.ld_x = a.ld_w = a.ld_dx = a.ld_dw = 16
    a.loss, a.lse, a.total = base + 0x20000, base + 0x21000, base + 0x22000
    a.dx, a.dw = base + 0x30000, base + 0x40000
    a.x_dtype = a.w_dtype = a.dx_dtype = a.dw_dtype = capi.DMUON_DTYPE_BF16
    a.target_dtype = capi.DMUON_INDEX_I64
    a.logit_scale = a.grad_scale = 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BASE = 0x10000000
CE_BAD = [
    ("ERR_SHAPE", dict(n_tokens=-1)), ("ERR_SHAPE", dict(n_tokens=1 << 31)), ("ERR_SHAPE", dict(vocab=0)),
    ("ERR_SHAPE", dict(vocab=(1 << 24) + 1)), ("ERR_SHAPE", dict(dim=0)), ("ERR_SHAPE", dict(ld_x=15)),
    ("ERR_SHAPE", dict(ld_w=15)), ("ERR_SHAPE", dict(ld_dx=15)), ("ERR_SHAPE", dict(ld_dw=15)),
    ("ERR_INVALID_ARG", dict(x=None)), ("ERR_INVALID_ARG", dict(w=None)), ("ERR_INVALID_ARG", dict(targets=None)),
    ("ERR_INVALID_ARG", dict(loss=None, lse=None, total=None, dx=None, dw=None)),
    ("ERR_INVALID_ARG", dict(logit_scale=0.0)), ("ERR_INVALID_ARG", dict(logit_scale=-1.0)),
    ("ERR_INVALID_ARG", dict(logit_scale=float("nan"))), ("ERR_INVALID_ARG", dict(logit_scale=float("inf"))),
    ("ERR_INVALID_ARG", dict(grad_scale=float("nan"))), ("ERR_INVALID_ARG", dict(flags=4)),
    ("ERR_DTYPE", dict(x_dtype=0)), ("ERR_DTYPE", dict(w_dtype=0)), ("ERR_DTYPE", dict(dx_dtype=2)),
    ("ERR_DTYPE", dict(dw_dtype=-1)), ("ERR_DTYPE", dict(target_dtype=2)),
    # written memory shared with anything else
    ("ERR_INVALID_ARG", dict(dx=BASE)), ("ERR_INVALID_ARG", dict(dw=BASE + 0x1000 + 100)),
    ("ERR_INVALID_ARG", dict(loss=BASE + 0x21000)), ("ERR_INVALID_ARG", dict(total=BASE + 0x30000 + 126)),
    ("ERR_INVALID_ARG", dict(lse=BASE + 0x10000 + 16)),
    # not on their elements' boundaries
    ("ERR_INVALID_ARG", dict(x=BASE + 1)), ("ERR_INVALID_ARG", dict(targets=BASE + 0x10004)),
    ("ERR_INVALID_ARG", dict(loss=BASE + 0x20002)), ("ERR_INVALID_ARG", dict(dw=BASE + 0x40002, dw_dtype=0)),
    ("ERR_INVALID_ARG", dict(weights=BASE + 0x50001)),
]


@pytest.mark.parametrize("status, kw", CE_BAD, ids=lambda v: str(v)[:40])
def test_cross_entropy_refusals(mos, status, kw):
    capi = mos.capi
    ctx = mos.dmuon_context_create(0)
    try:
        with pytest.raises(mos.DmuonError) as e:
            mos.dmuon_cross_entropy(ctx, ce_args(capi, **kw), 0)
        assert e.value.status == getattr(capi, "DMUON_" + status), (kw, e.value)
        assert "cross_entropy" in str(e.value)
    finally:
        mos.dmuon_context_destroy(ctx)


def embed_args(capi, **kw):
    a = capi.DmuonEmbed()
    a.n_tokens, a.vocab, a.dim = 4, 100, 16
    a.ids, a.table, a.rows = BASE, BASE + 0x1000, BASE + 0x10000
    a.ld_table = a.ld_rows = 16
    a.id_dtype = capi.DMUON_INDEX_I32
    a.table_dtype, a.row_dtype = capi.DMUON_DTYPE_F32, capi.DMUON_DTYPE_BF16
    a.scale = 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


EMBED_BAD = [
    ("ERR_SHAPE", dict(n_tokens=-1)), ("ERR_SHAPE", dict(vocab=0)), ("ERR_SHAPE", dict(dim=0)),
    ("ERR_SHAPE", dict(dim=(1 << 20) + 1)), ("ERR_SHAPE", dict(ld_table=15)), ("ERR_SHAPE", dict(ld_rows=15)),
    ("ERR_INVALID_ARG", dict(ids=None)), ("ERR_INVALID_ARG", dict(table=None)), ("ERR_INVALID_ARG", dict(rows=None)),
    ("ERR_INVALID_ARG", dict(scale=float("inf"))), ("ERR_INVALID_ARG", dict(flags=2)),
    ("ERR_DTYPE", dict(id_dtype=2)), ("ERR_DTYPE", dict(table_dtype=2)), ("ERR_DTYPE", dict(row_dtype=3)),
    ("ERR_INVALID_ARG", dict(rows=BASE + 0x1000 + 64)),
    ("ERR_INVALID_ARG", dict(ids=BASE + 2)), ("ERR_INVALID_ARG", dict(table=BASE + 0x1002)),
    ("ERR_INVALID_ARG", dict(rows=BASE + 0x10001)),
]


@pytest.mark.parametrize("entry", ["dmuon_embed_forward", "dmuon_embed_backward"])
@pytest.mark.parametrize("status, kw", EMBED_BAD, ids=lambda v: str(v)[:40])
def test_embed_refusals(mos, entry, status, kw):
    capi = mos.capi
    ctx = mos.dmuon_context_create(0)
    try:
        with pytest.raises(mos.DmuonError) as e:
            getattr(mos, entry)(ctx, embed_args(capi, **kw), 0)
        assert e.value.status == getattr(capi, "DMUON_" + status), (kw, e.value)
    finally:
        mos.dmuon_context_destroy(ctx)


def test_refusals_of_null_context_and_forward_flags(mos):
    capi = mos.capi
    with pytest.raises(mos.DmuonError) as e:
        mos.dmuon_cross_entropy(None, ce_args(capi), 0)
    assert e.value.status == capi.DMUON_ERR_INVALID_ARG
    lib = mos.load_library()
    ctx = mos.dmuon_context_create(0)
    try:
        assert lib.dmuon_cross_entropy(ctx, None, None) == capi.DMUON_ERR_INVALID_ARG
        a = embed_args(capi, flags=capi.DMUON_EMBED_ADD)
        assert lib.dmuon_embed_forward(ctx, ctypes.byref(a), None) == capi.DMUON_ERR_INVALID_ARG
    finally:
        mos.dmuon_context_destroy(ctx)


@pytest.mark.parametrize("flags", [16, 1 | 2 | 8 | 32, 1 << 31])
def test_cross_entropy_refuses_flags_it_does_not_know(mos, flags):
    ctx = mos.dmuon_context_create(0)
    try:
        with pytest.raises(mos.DmuonError) as e:
            mos.dmuon_cross_entropy(ctx, ce_args(mos.capi, flags=flags), 0)
        assert e.value.status == mos.capi.DMUON_ERR_INVALID_ARG and "flag" in str(e.value)
    finally:
        mos.dmuon_context_destroy(ctx)


def test_block_limit_key(mos):
    capi = mos.capi
    ctx = mos.dmuon_context_create(0)
    try:
        mos.dmuon_context_set_tuning(ctx, 14, 1)
        mos.dmuon_context_set_tuning(ctx, 14, 65536)
        for value in (0, -1, 65537):
            with pytest.raises(mos.DmuonError) as e:
                mos.dmuon_context_set_tuning(ctx, 14, value)
            assert e.value.status == capi.DMUON_ERR_INVALID_ARG
    finally:
        mos.dmuon_context_destroy(ctx)


def test_python_wrapper_checks(mos):
    import torch

    ops = mos.VocabOps(0)
    cpu = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ops.cross_entropy(cpu, cpu, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        ops.embed(torch.zeros(4, dtype=torch.int64), cpu, cpu)
    ops.close()


# Column ranges of one buffer at 80 elements (160 bytes) a row: x 16 wide at column 0.
INTERLEAVED = [
    (True, dict(ld_x=80, ld_dx=80, dx=BASE + 32)), (True, dict(ld_x=80, ld_dx=80, dx=BASE + 128)),
    (False, dict(ld_x=80, ld_dx=80, dx=BASE + 30)), (False, dict(ld_x=80, ld_dx=80, dx=BASE + 130)),
    (False, dict(ld_x=80, ld_dx=80, dx=BASE + 160)), (False, dict(ld_x=80, ld_dx=80, dx=BASE + 160 * 3 + 30)),
    (True, dict(ld_x=80, ld_dx=80, dx=BASE + 160 * 3 + 32)), (True, dict(ld_x=80, ld_dx=40, dx_dtype=0, dx=BASE + 32)),
    (False, dict(ld_x=80, ld_dx=40, dx_dtype=0, dx=BASE + 100)),
    (False, dict(ld_x=80, ld_dx=40, dx=BASE + 32)),  # other pitches: by their spans
    (True, dict(ld_x=80, loss=BASE + 32)), (True, dict(ld_x=80, loss=BASE + 160 + 144)), (False, dict(ld_x=80, loss=BASE + 148)),
    (False, dict(ld_x=80, loss=BASE - 12)), (True, dict(ld_x=80, loss=BASE - 16)), (False, dict(ld_x=80, total=BASE + 160 + 28)),
]


@pytest.mark.parametrize("fine, kw", INTERLEAVED, ids=lambda v: str(v)[:60])
def test_column_ranges_of_one_buffer(mos, fine, kw):
    # Without a device a call that passes its checks ends at that; a refusal names the overlap.
    ctx = mos.dmuon_context_create(99)
    try:
        with pytest.raises(mos.DmuonError) as e:
            mos.dmuon_cross_entropy(ctx, ce_args(mos.capi, **kw), 0)
        assert ("overlaps" not in str(e.value)) == fine, (kw, e.value)
    finally:
        mos.dmuon_context_destroy(ctx)


def test_sync_waits_for_its_own_devices_stream(mos, monkeypatch):
    from matrix_optimizer_step_gb300 import vocab

    ops = mos.VocabOps(1)
    seen = []
    monkeypatch.setattr(vocab, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(vocab.capi, "dmuon_sync", lambda ctx, stream=None: seen.append(stream))
    ops.sync()
    ops.sync(7)
    assert seen == [1001, 7]
    ops.close()


def test_overlapped_kernels_read_with_ordered_loads():
    # These kernels' blocks are resident while the kernel before them still writes; the read-only path is for memory
    # that nothing writes during a kernel's life.
    import os
    import re

    here = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "matrix_optimizer_step_gb300", "csrc")
    for name in ("vocab.h", "vocab.cu", "k_embed.cu", "k_vocab_ce.cu", "k_vocab_gemm.cu", "k_vocab_thin.cu"):
        with open(os.path.join(here, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__ldcg\s*\(", code), name
