"""Gradient operators without a GPU: the oracle, and every argument check of the
C entry points and of their callers (all refusals happen on the host)."""

import math

import pytest

from oracle import grads as ograds


@pytest.fixture(scope="module")
def mos():
    import matrix_optimizer_step_gb300 as m
    from matrix_optimizer_step_gb300 import build

    build.build()
    m.load_library()
    return m


def test_oracle_norms():
    norm, each = ograds.norms([[3.0, 4.0], [], [1e300, 0.0]])
    assert each == [5.0, 0.0, 1e300] and norm == 1e300
    assert ograds.factor(2.0, 1.0) == 1 / (2 + 1e-6) and ograds.factor(0.0, 1.0) == 1.0
    assert ograds.factor(math.inf, 1.0) == 0.0 and ograds.factor(math.inf, math.inf) == 1.0
    assert math.isnan(ograds.factor(math.nan, 1.0))


BASE = 0x10000000  # plausible, never dereferenced: every case here is refused on the host
NORM, COEF, NORMS = BASE + 0x100000, BASE + 0x100010, BASE + 0x100020
INV = "ERR_INVALID_ARG"


class _At:
    """A pointer as capi._ptr reads one."""

    def __init__(self, p):
        self.p = p

    def data_ptr(self):
        return self.p


def grad_list(capi, **kw):
    a = (capi.DmuonGrad * 3)()
    for i in range(3):
        a[i] = capi.DmuonGrad(1000, BASE + 0x10000 * i, BASE + 0x10000 * i, i % 2, i % 2)
    for k, v in kw.items():
        setattr(a[1], k, v)
    return a


@pytest.fixture()
def ctx(mos):
    c = mos.dmuon_context_create(0)
    yield c
    mos.dmuon_context_destroy(c)


GRAD_BAD = [
    ("ERR_SHAPE", dict(numel=-1), {}), ("ERR_SHAPE", dict(numel=(1 << 40) + 1), {}),
    ("ERR_DTYPE", dict(grad_dtype=2), {}), ("ERR_DTYPE", dict(out_dtype=-1), {}),
    (INV, dict(grad=None), {}), (INV, dict(out=None), {}),
    (INV, dict(grad=BASE + 0x10001, out=BASE + 0x10001), {}), (INV, dict(out=BASE + 0x50001), {}),
    (INV, {}, dict(max_norm=0.0)), (INV, {}, dict(max_norm=-1.0)), (INV, {}, dict(max_norm=float("nan"))),
    (INV, {}, dict(n=-1)), (INV, {}, dict(array=None)), ("ERR_SHAPE", {}, dict(n=(1 << 24) + 1)),
]


@pytest.mark.parametrize("status, kw, call", GRAD_BAD, ids=lambda v: str(v)[:40])
def test_clip_grads_refusals(mos, ctx, status, kw, call):
    capi = mos.capi
    array = call.get("array", grad_list(capi, **kw))
    with pytest.raises(mos.DmuonError) as e:
        mos.dmuon_clip_grads(ctx, array, call.get("n", 3), call.get("max_norm", 1.0), _At(NORM), _At(NORMS), _At(COEF), 0)
    assert e.value.status == getattr(capi, "DMUON_" + status), (kw, e.value)
    assert "clip_grads" in str(e.value)
    if "out" not in kw and "out_dtype" not in kw:
        with pytest.raises(mos.DmuonError) as e:
            mos.dmuon_grad_norm(ctx, array, call.get("n", 3), call.get("max_norm", 1.0), _At(NORM), None, _At(COEF), 0)
        assert e.value.status == getattr(capi, "DMUON_" + status) and "grad_norm" in str(e.value)


OVERLAPS = [dict(out=BASE + 0x10002), dict(out=BASE), dict(out_dtype=0, grad_dtype=1), dict(grad=BASE + 100, out=BASE + 100),
            dict(out=NORM - 1996), dict(out=COEF - 1998), dict(out=NORMS)]


@pytest.mark.parametrize("kw", OVERLAPS, ids=str)
def test_clip_grads_overlaps(mos, ctx, kw):
    capi = mos.capi
    with pytest.raises(mos.DmuonError) as e:
        mos.dmuon_clip_grads(ctx, grad_list(capi, **kw), 3, 1.0, _At(NORM), _At(NORMS), _At(COEF), 0)
    assert e.value.status == capi.DMUON_ERR_INVALID_ARG and "overlaps" in str(e.value), (kw, e.value)


def test_lists_that_share_nothing_pass_the_overlap_check(mos, ctx):
    # Gradients may share memory with one another where nothing is written; these calls end at the device, or at
    # pointers that it cannot reach.
    capi = mos.capi
    for call in (lambda: mos.dmuon_clip_grads(ctx, grad_list(capi), 3, 1.0, _At(NORM), _At(NORMS), _At(COEF), 0),
                 lambda: mos.dmuon_grad_norm(ctx, grad_list(capi, grad=BASE + 2), 3, 1.0, _At(NORM), None, None, 0)):
        with pytest.raises(mos.DmuonError) as e:
            call()
        assert "overlaps" not in str(e.value)


def test_other_refusals(mos, ctx):
    capi = mos.capi
    for call in (lambda: mos.dmuon_grad_norm(ctx, grad_list(capi), 3, 1.0, None, None, None, 0),
                 lambda: mos.dmuon_grad_norm(ctx, grad_list(capi), 3, 1.0, _At(NORM + 2), None, None, 0),
                 lambda: mos.dmuon_scale_grads(ctx, grad_list(capi), 3, None, 0),
                 lambda: mos.dmuon_scale_grads(ctx, grad_list(capi), 3, _At(BASE + 16), 0),
                 lambda: mos.dmuon_clip_grads(None, grad_list(capi), 3, 1.0, None, None, None, 0)):
        with pytest.raises(mos.DmuonError) as e:
            call()
        assert e.value.status == capi.DMUON_ERR_INVALID_ARG, e.value


@pytest.mark.parametrize("at", [BASE + 2, BASE + 0x1000, BASE + 0x1000 + 3996, BASE + 0x3000 - 4, BASE + 0x4000])
def test_scaled_steps_refuse_their_own_memory(mos, ctx, at):
    capi = mos.capi
    v, m = capi.DmuonVector(), capi.DmuonMatrix()
    v.numel, v.grad, v.grad_dtype = 1000, BASE + 0x8000, 0
    v.master, v.exp_avg, v.exp_avg_sq, v.param_bf16 = BASE + 0x1000, BASE + 0x2060, BASE + 0x3000, BASE + 0x4000
    m.rank, m.grad_dtype, m.grad = 2, 0, BASE + 0x8000
    m.shape[0], m.shape[1] = 10, 100
    m.master, m.momentum, m.param_bf16 = BASE + 0x1000, BASE + 0x2060, BASE + 0x4000
    for call in (lambda: mos.dmuon_adamw_step_scaled(ctx, capi.descriptor_array([v], capi.DmuonVector), 0.1, 0.9, 0.9, 0.1, 0.0, 1, _At(at), 0),
                 lambda: mos.dmuon_muon_step_scaled(ctx, capi.descriptor_array([m], capi.DmuonMatrix), 0.1, 0.9, 0.0, 5, 1.0, 1.0, 1.0, _At(at), 1, 0)):
        with pytest.raises(mos.DmuonError) as e:
            call()
        assert e.value.status == capi.DMUON_ERR_INVALID_ARG and "grad_scale" in str(e.value), e.value


def test_python_refusals(mos):
    import torch

    grads, owner = mos.GradOps(0), mos.OwnerStep(0)
    with pytest.raises(TypeError):
        grads.register([torch.zeros(3)])  # not on the device
    with pytest.raises(ValueError):
        grads.register([], [torch.zeros(3)])
    empty = grads.register([])
    with pytest.raises(ValueError):
        grads.norm(empty, coef=torch.zeros(1))
    with pytest.raises(TypeError):
        grads.clip(empty, 1.0, norm=torch.zeros(1))
    with pytest.raises(RuntimeError):
        owner.grad_norm()
    with pytest.raises(RuntimeError):
        owner.step(None, None, stream=object())
    with pytest.raises(RuntimeError):
        owner.step(dict(lr=0.1, momentum=0.9, wd=0.0), None, stream=object())
    owner._mats = object()
    with pytest.raises(ValueError):
        owner.step(dict(lr=0.1, momentum=0.9, wd=0.0, grad_scale=1), None, stream=object(), max_norm=1.0)
    with pytest.raises(ValueError):
        owner.step(dict(lr=0.1, momentum=0.9, wd=0.0), None, stream=object(), norm=torch.zeros(1))


class _Stream:
    def wait_event(self, event):
        pass


class _Event:
    def record(self, stream):
        pass


def test_a_clipped_step_has_a_factor_of_its_own(mos, monkeypatch):
    # The Muon route on one stream and the AdamW route on another share no tensor, so either's norm may be written
    # while the other's step has yet to read its factor.
    import torch

    from matrix_optimizer_step_gb300 import optim

    taken, calls = [], []
    monkeypatch.setattr(optim, "empty_on", lambda stream, *a, **kw: taken.append((stream, torch.empty(1))) or taken[-1][1])
    step = optim.OwnerStep(0)
    step._mats = step._vecs = ()
    step._side, step._ev_fork, step._ev_join = _Stream(), _Event(), _Event()
    monkeypatch.setattr(step, "_grad_norm", lambda muon, adamw, max_norm, norm, norms, coef, stream: calls.append((stream, coef)))
    monkeypatch.setattr(step, "muon_step", lambda stream, grad_scale: calls.append((stream, grad_scale)))
    monkeypatch.setattr(step, "adamw_step", lambda stream, grad_scale: calls.append((stream, grad_scale)))
    streams = [_Stream() for _ in range(3)]
    step.step({}, None, stream=streams[0], max_norm=1.0)
    step.step(None, {}, stream=streams[1], max_norm=1.0)
    step.step({}, {}, stream=streams[2], max_norm=1.0)
    step.close()
    assert [s for s, _ in taken] == streams
    where = {id(t): i for i, (_, t) in enumerate(taken)}
    assert [where[id(t)] for _, t in calls] == [0, 0, 1, 1, 2, 2, 2]
    assert len({t.data_ptr() for _, t in taken}) == 3
