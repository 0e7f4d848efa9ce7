"""Vocabulary operators on the GPU, cases that an earlier form of them answered wrongly.

Bounds are those of test_gpu_vocab.py (U = 2^-8 and F = 2^-24, the unit roundoffs of bf16 and fp32), each
with what the case adds to them.
"""

import numpy as np
import pytest
import torch

from oracle import vocab as ovocab
from test_gpu_vocab import DEV, F, U, f64, inputs, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops(cuda_lib):
    o = cuda_lib.VocabOps(0)
    yield o
    o.close()


# -------------------------------------------------- d logits in two halves

def fine_bounds(x, w, t, a, grad_scale):
    """dx, dw in float64, and how far off they may be with fp32 outputs and d logits in two bf16 halves: of a
    d logit (dz) the remainder's rounding U^2 |dz|, of a probability its log's step and the logit's error, as in
    check_ce; then the product's fp32 sums (twice as long: hi and lo) and one rounding."""
    n, d = x.shape
    v = w.shape[0]
    X, W, T = f64(x), f64(w), t.cpu().numpy()
    A = f64(a)
    r = ovocab.cross_entropy(X, W, T, A, grad_scale=grad_scale)
    counted = T >= 0
    X = np.where(counted[:, None], X, 0.0)
    ez = (d / 16 + 8) * 4 * F * float((np.abs(X) @ np.abs(W).T).max())
    coef = np.where(counted, A, 0.0)
    coef = grad_scale * coef / coef.sum()
    adz = np.abs(r["dz"])
    p = adz.copy()
    rows = np.arange(n)[counted]
    p[rows, T[counted]] = coef[counted] - p[rows, T[counted]]
    ep = 2 * ez + np.log(2) / 2048 + 32 * F
    edz = adz * U * U + p * ep + coef[:, None] * 2.0 ** -60
    edz[rows, T[counted]] += 8 * F * coef[counted]
    out = {}
    for name, k, E, A_, B in (("dx", 2 * v, edz, adz, np.abs(W)), ("dw", 2 * n, edz.T, adz.T, np.abs(X))):
        e = E @ B + (k / 16 + 8) * 4 * F * (A_ @ B)
        out[name] = (r[name], e + F * (np.abs(r[name]) + e) + 1e-38)
    return out


@pytest.mark.parametrize("n, v, d, block_mib", [(129, 513, 72, 0), (300, 5003, 136, 0), (257, 1030, 200, 0), (700, 777, 1001, 0),
                                                (700, 5003, 136, 1), (1100, 600, 264, 0), (2100, 130, 40, 0)])
@pytest.mark.parametrize("add", [False, True])
def test_fine_gradients(cuda_lib, n, v, d, block_mib, add):
    ops = cuda_lib.VocabOps(0)
    if block_mib:
        ops.set_tuning(14, block_mib)  # several passes
    x, w, t, a = (q.to(DEV) for q in inputs(n, v, d, seed=n + v))
    base = torch.randn(v, d, device=DEV) * 1e-3
    want = fine_bounds(x, w, t, a, 0.5)
    err = {}
    for fine in (True, False):
        dx, dw = torch.full((n, d), 7.0, device=DEV), base.clone()
        ops.cross_entropy(x, w, t, weights=a, grad_scale=0.5, dx=dx, dw=dw, accumulate_dw=add, fine_grads=fine)
        ops.sync()
        for name, got in (("dx", dx), ("dw", dw)):
            ref, tol = want[name]
            if name == "dw" and add:
                ref, tol = ref + f64(base), tol + 4 * F * (np.abs(ref) + np.abs(f64(base)))
            if fine:
                within(got, ref, tol, name)
            err[name, fine] = np.linalg.norm(f64(got) - ref)
    # What the option is for: dw's error is that of its targets' d logits, which one half rounds to U / 2.
    assert err["dw", True] < 0.5 * err["dw", False], err
    ops.close()


def test_fine_gradients_of_few_tokens_are_the_same(ops):
    # Up to 128 tokens come in two halves anyway.
    x, w, t, a = (q.to(DEV) for q in inputs(128, 900, 64, seed=3))
    got = []
    for fine in (False, True):
        dx, dw = torch.empty(128, 64, device=DEV), torch.empty(900, 64, device=DEV)
        ops.cross_entropy(x, w, t, weights=a, dx=dx, dw=dw, fine_grads=fine)
        got.append((dx, dw))
    ops.sync()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ------------------------------------------------------------------- streams

def busy(stream, ms=60):
    """About `ms` of work on `stream` (a kernel of torch's that counts clock cycles)."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(ms * 2.0e6))


@pytest.mark.parametrize("busy_default", [True, False])
def test_first_call_of_a_handle_on_a_side_stream(cuda_lib, busy_default):
    # The handle's counters and error word are cleared by its first call.  That call's kernels, on a stream that does
    # not wait for the default one, must not run before the clearing, whatever the default stream has to do.
    # More than 76 pairs' worth of tiles of 32 k-blocks: they are drawn from the counters.
    n, v, d = 300, 22000, 2056
    x, w, t, a = (q.to(DEV) for q in inputs(n, v, d, seed=21))
    bad = t.clone()
    bad[5] = v
    s = torch.cuda.Stream()
    keys = ("loss", "lse", "total", "dx", "dw")

    def outputs():
        return dict(loss=torch.full((n,), 7.0, device=DEV), lse=torch.full((n,), 7.0, device=DEV),
                    total=torch.full((1,), 7.0, device=DEV), dx=torch.full_like(x, 7.0), dw=torch.full_like(w, 7.0))

    for targets in (t, bad):
        ops = cuda_lib.VocabOps(0)
        first, second = outputs(), outputs()
        torch.cuda.synchronize()
        if busy_default:
            busy(torch.cuda.default_stream())
        ops.cross_entropy(x, w, targets, weights=a, stream=s, **first)
        if targets is bad:  # the report is not cleared away either
            with pytest.raises(cuda_lib.DmuonError):
                ops.sync(s)
        else:
            ops.sync(s)
        torch.cuda.synchronize()
        ops.cross_entropy(x, w, targets, weights=a, **second)
        torch.cuda.synchronize()
        assert all(torch.equal(first[k], second[k]) for k in keys)
        ops.close()


@pytest.mark.parametrize("n, v, d", [(64, 900, 64), (300, 3000, 264), (2100, 1500, 72), (5000, 700, 40)])
def test_calls_that_feed_one_another(ops, n, v, d):
    # A call's kernels may be resident while the one before still writes what they read: ids, rows and gradients go
    # from call to call, other ones each time and in the same memory, against the same calls one at a time.
    steps = [tuple(q.to(DEV) for q in inputs(n, v, d, seed=30 + k)) for k in range(4)]
    w = steps[0][1]
    ids, targets = torch.empty(n, dtype=torch.int64, device=DEV), torch.empty(n, dtype=torch.int64, device=DEV)
    weights, x, dx = torch.empty(n, device=DEV), torch.empty(n, d, device=DEV, dtype=torch.bfloat16), torch.empty(n, d, device=DEV)
    out = {}
    for wait in (True, False):
        out[wait] = []
        dw = torch.empty(v, d, device=DEV)
        for k, (_, _, t, a) in enumerate(steps * 3):
            ids.copy_(t.roll(1))
            targets.copy_(t)
            weights.copy_(a)
            for call in (lambda: ops.embed(ids, w, x, scale=3.0),
                         lambda: ops.cross_entropy(x, w, targets, weights=weights, dx=dx, dw=dw),
                         lambda: ops.embed_grad(ids, dx, dw, accumulate=True),
                         lambda: out[wait].append((dx.clone(), dw.clone()))):
                call()
                if wait:
                    torch.cuda.synchronize()
    ops.sync()
    for a, b in zip(out[True], out[False]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_one_stream_handle_in_two_threads(cuda_lib):
    # cudaStreamPerThread (handle 2) is another stream in each thread; calls on the two share the context's scratch
    # and have to wait for one another.
    import threading

    per_thread = 2
    ops = cuda_lib.VocabOps(0)
    sets = [tuple(q.to(DEV) for q in inputs(n, v, d, seed=n)) for n, v, d in ((500, 3000, 200), (300, 5000, 264))]
    want, got = [], []
    for x, w, t, a in sets:
        for to in (want, got):
            to.append(dict(loss=torch.empty(x.shape[0], device=DEV), dx=torch.empty_like(x), dw=torch.empty_like(w)))
        ops.cross_entropy(x, w, t, weights=a, **want[-1])
    ops.sync()
    torch.cuda.synchronize()

    def call(k, first, then):
        if first:
            busy(torch.cuda.ExternalStream(per_thread, device=0), 30)
        x, w, t, a = sets[k]
        ops.cross_entropy(x, w, t, weights=a, stream=per_thread, **got[k])
        if then is not None:
            then()
        torch.cuda.ExternalStream(per_thread, device=0).synchronize()

    def other():
        # While the first thread's call still waits behind its stream's work.
        th = threading.Thread(target=call, args=(1, False, None))
        th.start()
        th.join()

    first = threading.Thread(target=call, args=(0, True, other))
    first.start()
    first.join()
    torch.cuda.synchronize()
    ops.sync()
    for a, b in zip(want, got):
        assert all(torch.equal(a[k], b[k]) for k in a)
    ops.close()


@pytest.mark.parametrize("what", ["embed", "loss"])
@pytest.mark.parametrize("as_handle", [False, True])
def test_results_that_the_wrapper_allocates_belong_to_the_stream(ops, what, as_handle):
    # Memory that the current stream has freed but is still to write must not become the result of a call on another.
    n, v, d = 60000, 500, 8
    x, w, t, _ = (q.to(DEV) for q in inputs(n, v, d, seed=5))

    def call(stream=None):
        if what == "embed":
            return ops.embed(t, w, stream=stream)
        return ops.cross_entropy(x, w, t, stream=stream)

    want = call().clone()
    s = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        old = torch.empty_like(want)
        busy(torch.cuda.current_stream(), 20)
        old.fill_(3.0)
        del old
        got = call(s.cuda_stream if as_handle else s)
        with torch.cuda.stream(s):
            same = torch.equal(got, want)
        torch.cuda.synchronize()
        assert same and torch.equal(got, want)
    ops.sync()


def test_lookup_on_the_default_streams_handle(ops):
    # Handle 0 is the default stream, whichever is current.
    w = torch.randn(50, 16, device=DEV)
    t = torch.arange(40, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = ops.embed(t, w, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, w[:40])


@pytest.mark.parametrize("ids, table", [([1, 2], None), (None, torch.zeros(4)), (None, [[1.0]])])
def test_lookup_without_an_output_refuses_before_it_allocates(ops, ids, table):
    good = torch.zeros(4, 16, device=DEV)
    index = torch.zeros(2, dtype=torch.int64, device=DEV)
    if isinstance(table, torch.Tensor):
        table = table.to(DEV)
    with pytest.raises((TypeError, ValueError)):
        ops.embed(index if ids is None else ids, good if table is None else table)


# ------------------------------------------------------------ logits as summed

@pytest.mark.parametrize("d", [4096, 8192])
@pytest.mark.parametrize("n", [3, 40, 70, 300])
def test_sparse_rows_keep_the_digits_of_certain_tokens(ops, n, d):
    # One-hot hidden states: every logit is one product, exact in fp32, whatever the width.  Column k's target
    # stands at 40, the next entry at 20 to 30, so the loss is exp(that - 40) and more, relatively off by the
    # absolute error of the competitor's logit: the rounding of the scale and of z - m at 60 octaves (60 ln 2 F
    # each), the exponentials, the additions and the last steps (80 F, as for narrow heads).
    v, used = 500, 8
    g = torch.Generator(device=DEV).manual_seed(n)
    at = torch.randperm(d, generator=g, device=DEV)[:used]
    w = torch.zeros(v, d, device=DEV, dtype=torch.bfloat16)
    k = torch.arange(used, device=DEV)
    w[:, at] = (torch.rand(v, used, generator=g, device=DEV) * 4 - 2).to(torch.bfloat16)
    w[10 * k, at] = 40.0
    w[10 * k + 1, at] = (20 + 10 * k / 7).to(torch.bfloat16)
    which = torch.arange(n, device=DEV) % used
    x = torch.zeros(n, d, device=DEV, dtype=torch.bfloat16)
    x[torch.arange(n, device=DEV), at[which]] = 1.0
    t = 10 * which
    loss, scores, dw = torch.empty(n, device=DEV), torch.empty(n, device=DEV), torch.empty(v, d, device=DEV)
    ops.cross_entropy(x, w, t, loss=loss, dw=dw)
    ops.cross_entropy(x, w, t, loss=scores)
    ops.sync()
    z = w.double()[:, at].T[which]
    top = z.gather(1, t[:, None])
    want = torch.log1p(torch.exp(z - top).scatter(1, t[:, None], 0.0).sum(1))
    tol = (2 * 60 * np.log(2) + 80) * F
    for got in (loss, scores):
        within(f64(got), f64(want), tol * f64(want), "loss")


@pytest.mark.parametrize("n", [16, 300])
@pytest.mark.parametrize("d", [1024, 4096, 8192])
def test_dense_log_sums_are_not_lifted(ops, n, d):
    # The matrix instruction's running sum may truncate, towards zero: 2 F of the sum at most for each 16 products.
    # Rows that lean on a few of w's rows have log-sums that are these logits', whose sums grow steadily: on average
    # a log-sum may come out lower by that, and higher by no more than the roundings outside of the product.
    v = 2000
    g = torch.Generator(device=DEV).manual_seed(n + d)
    w = (torch.randn(v, d, generator=g, device=DEV) * (1.3 / d ** 0.5)).to(torch.bfloat16)
    on = torch.randint(0, v, (n,), generator=g, device=DEV)
    x = (torch.randn(n, d, generator=g, device=DEV) * 0.1 + 12.0 * w[on].float()).to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    lse = torch.empty(n, device=DEV)
    ops.cross_entropy(x, w, t, lse=lse)
    ops.sync()
    z = x.double() @ w.double().T
    want = torch.logsumexp(z, 1)
    off = float((lse.double() - want).mean())
    top = float(z.max(1).values.mean())
    assert off <= 8 * F * top, (off, top)
    assert off >= -(d / 16) * 2 * F * top - 8 * F * top, (off, top)


@pytest.mark.parametrize("n", [3, 70, 300])
@pytest.mark.parametrize("level", [-200.0, -5.0])
def test_blocks_without_finite_logits(ops, n, level):
    # 256 entries of every row are -inf (ids ruled out by w), the others far below zero, or not.  Each logit is a sum
    # of two products, exact in fp32; lse and loss: the scale's and m's roundings and the last steps, 8 F |lse| each
    # as elsewhere, the exponentials and additions 64 F.  The target of row 0 is itself ruled out.
    v, d = 1000, 16
    g = torch.Generator(device=DEV).manual_seed(n)
    w = torch.zeros(v, d, device=DEV, dtype=torch.bfloat16)
    w[:, 0] = level
    w[128:384, 0] = float("-inf")
    w[:, 1] = torch.randint(-16, 17, (v,), generator=g, device=DEV).to(torch.bfloat16) / 8
    x = torch.zeros(n, d, device=DEV, dtype=torch.bfloat16)
    x[:, :2] = 1.0
    t = torch.randint(384, v, (n,), generator=g, device=DEV)
    t[0], t[1] = 200, -1
    for grads in (False, True):
        loss, lse, dw = torch.empty(n, device=DEV), torch.empty(n, device=DEV), torch.zeros(v, d, device=DEV)
        ops.cross_entropy(x, w, t, loss=loss, lse=lse, mean=False, **(dict(dw=dw) if grads else {}))
        ops.sync()
        z = w[:, 0].double() + w[:, 1].double()
        want = float(torch.logsumexp(z, 0))
        tol = (64 + 16 * abs(want)) * F
        counted = t >= 0
        assert bool(((lse[counted].double() - want).abs() <= tol).all()), (lse[:4], want)
        assert float(lse[1]) == 0 and float(loss[1]) == 0 and float(loss[0]) == float("inf")
        assert bool(((loss[2:].double() - (want - z[t[2:]])).abs() <= tol).all())
    p = torch.exp(z - want)
    counts = torch.bincount(t[counted], minlength=v).double()
    ref = p * float(counted.sum()) - counts
    # a probability's log is kept in steps of 2^-10 octaves, d logits as one bf16 (two up to 128 tokens), sums in fp32
    tol = (p * float(counted.sum()) + counts) * (np.log(2) / 2048 + U + (n + 64) * F) + 1e-30
    assert bool(((dw[:, 0].double() - ref).abs() <= tol).all())


# ------------------------------------------------------ column ranges of one buffer

@pytest.mark.parametrize("n, d, gap", [(300, 64, 0), (40, 40, 0), (300, 33, 3), (130, 72, 8)])
def test_column_ranges_of_one_buffer(ops, n, d, gap):
    # x and dx, w and dw, a table and its rows: the same bits as apart, and nothing between them written.
    v = 700
    x, w, t, a = (q.to(DEV) for q in inputs(n, v, d, seed=n + d))

    def apart():
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        loss = torch.empty(n, device=DEV)
        ops.cross_entropy(x, w, t, weights=a, loss=loss, dx=dx, dw=dw)
        return loss, dx, dw

    def together(left):
        out = []
        for q in (x, w):
            buf = torch.full((q.shape[0], 2 * d + 3 * gap), 3.0, device=DEV, dtype=torch.bfloat16)
            first, second = buf[:, gap:gap + d], buf[:, d + 2 * gap:2 * d + 2 * gap]
            first.copy_(q) if left else second.copy_(q)
            out.append((buf, first if left else second, second if left else first))
        (bx, xs, dx), (bw, ws, dw) = out
        loss = torch.empty(n, device=DEV)
        ops.cross_entropy(xs, ws, t, weights=a, loss=loss, dx=dx, dw=dw)
        ops.sync()
        assert torch.equal(xs, x) and torch.equal(ws, w)
        for buf in (bx, bw):
            for k in (0, d + gap, 2 * d + 2 * gap):
                assert bool((buf[:, k:k + gap] == 3).all())
        return loss, dx, dw

    want = apart()
    for left in (True, False):
        for p, q in zip(want, together(left)):
            # x and w start elsewhere in memory (copied or not), which moves no sum but the target's few lanes
            assert torch.allclose(p.float(), q.float(), rtol=2 * U, atol=1e-6), float((p.float() - q.float()).abs().max())
    buf = torch.full((v, 2 * d), 3.0, device=DEV)
    buf[:, :d] = w
    rows = buf[:n, d:]
    ids = t.clamp(min=0)
    ops.embed(ids, buf[:, :d], rows)
    ops.embed_grad(ids, rows, buf[:, :d])
    ops.sync()
    assert torch.equal(rows, w[ids].float()) and bool((buf[n:, d:] == 3).all())
    want = torch.zeros(v, d, dtype=torch.float64, device=DEV).index_add_(0, ids, rows.double())
    assert bool(((buf[:, :d].double() - want).abs() <= n * F * want.abs() + 1e-30).all())
    with pytest.raises(RuntimeError):
        ops.embed(ids, buf[:, :d], buf[:n, d - 1:2 * d - 1])


def test_a_capture_that_cannot_grow_the_scratch_loses_nothing(cuda_lib):
    # Memory cannot be had or freed while a stream is captured (in the default mode): the call is refused, and the
    # scratch that was there serves the calls after it.
    import ctypes

    cuda = ctypes.CDLL("libcuda.so.1")
    ops = cuda_lib.VocabOps(0)
    x, w, t, _ = (q.to(DEV) for q in inputs(1000, 60000, 16, seed=2))  # 120 MB of logs
    bx, bt = x.repeat(3, 1), t.repeat(3)
    out = dict(loss=torch.empty(1000, device=DEV), dx=torch.empty_like(x))
    big = dict(loss=torch.empty(3000, device=DEV), dx=torch.empty_like(bx))
    s = torch.cuda.Stream()
    ops.cross_entropy(x, w, t, **out)
    ops.sync()
    want = {k: q.clone() for k, q in out.items()}
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        assert cuda.cuStreamBeginCapture_v2(ctypes.c_void_p(s.cuda_stream), 0) == 0
        with pytest.raises(cuda_lib.DmuonError):
            ops.cross_entropy(bx, w, bt, stream=s, **big)
        graph = ctypes.c_void_p()
        cuda.cuStreamEndCapture(ctypes.c_void_p(s.cuda_stream), ctypes.byref(graph))
        assert not graph.value
        out["loss"].zero_()
        ops.cross_entropy(x, w, t, **out)
        ops.sync()
        assert all(torch.equal(want[k], out[k]) for k in want)
    assert torch.cuda.mem_get_info()[0] > free - (64 << 20)
    # The larger call then gives what it gives on a handle of its own.
    ops.cross_entropy(bx, w, bt, **big)
    ops.sync()
    other = cuda_lib.VocabOps(0)
    ref = {k: torch.empty_like(q) for k, q in big.items()}
    other.cross_entropy(bx, w, bt, **ref)
    other.sync()
    assert all(torch.equal(ref[k], big[k]) for k in ref)
    ops.close()
    other.close()
