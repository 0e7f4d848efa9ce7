"""User-facing wrapper of the vocabulary operators: embedding lookup, softmax
cross entropy and log probabilities over the output head, each with its gradient.

``VocabOps`` keeps a library context; its methods check and marshal torch
tensors, and everything runs in the CUDA library through the C ABI.  The
gradients have the dtypes ``OwnerStep.set_adamw`` takes, so an embedding table
or head goes from here straight to its AdamW step.
"""

from __future__ import annotations

import ctypes

import torch

from . import capi

_FLOATS = {torch.bfloat16: capi.DMUON_DTYPE_BF16, torch.float32: capi.DMUON_DTYPE_F32}
_BF16, _F32 = (torch.bfloat16,), (torch.float32,)
_INDEX = {torch.int32: capi.DMUON_INDEX_I32, torch.int64: capi.DMUON_INDEX_I64}

_Tensor = torch.Tensor


def _current_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# The handle alone where torch offers it (the stream object costs a microsecond).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def empty_on(stream, device, *shape, dtype):
    """Memory for a result that ``stream`` writes: torch's allocator gives a block out again in the order of the
    stream it was taken on, so it is taken on that one."""
    if stream is None:
        return torch.empty(shape, device=torch.device("cuda", device), dtype=dtype)
    handle = getattr(stream, "cuda_stream", stream)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)):
        return torch.empty(shape, device=torch.device("cuda", device), dtype=dtype)


class Ops:
    """A context on one GPU, and what its operators' handles have in common."""

    def __init__(self, device=0):
        self.device = int(device)
        self.ctx = capi.dmuon_context_create(self.device)
        self._lib = capi.load_library()

    def _list(self, t, name, dtypes, n):
        if not isinstance(t, _Tensor) or t.get_device() != self.device or t.dtype not in dtypes:
            self._refuse(t, name, dtypes)
        if t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name}: expected {n} contiguous elements")
        return t.data_ptr()

    def _refuse(self, t, name, dtypes):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != self.device:
            raise TypeError(f"{name} must be a tensor on cuda:{self.device}")
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")

    def _empty(self, stream, *shape, dtype):
        return empty_on(stream, self.device, *shape, dtype=dtype)

    def _stream(self, stream):
        return _raw_stream(self.device) if stream is None else getattr(stream, "cuda_stream", stream)

    def _call(self, fn, args, stream):
        status = fn(self.ctx, ctypes.byref(args), self._stream(stream))
        if status:
            capi._check(status)

    # ---------------------------------------------------------------- misc
    def sync(self, stream=None):
        """Wait for ``stream`` (None: the handle's device's current one) and raise
        DmuonError for device-side errors."""
        capi.dmuon_sync(self.ctx, _raw_stream(self.device) if stream is None else stream)

    def set_tuning(self, key, value):
        """One tuning key of this context (dmuon_context_set_tuning)."""
        capi.dmuon_context_set_tuning(self.ctx, key, value)

    def kernel_launches(self):
        return capi.dmuon_kernel_launches(self.ctx)

    def close(self):
        if self.ctx is not None:
            capi.dmuon_context_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class VocabOps(Ops):
    """Embedding, cross entropy and log probabilities on one GPU.

    Matrices are (rows, width) tensors with contiguous rows (any row pitch);
    lists are contiguous.  Work is enqueued on ``stream`` (a torch stream or
    handle; None: the current one) and returns without waiting; ``sync``
    reports device-side errors, an id past the vocabulary among them.

    No autograd graph is recorded, whether tensors require gradients or not: a
    result is plain data, and gradients are the outputs asked for (``dx`` goes on
    as ``x.backward(dx)``).  The handle's scratch comes from CUDA, not from
    torch's allocator, and is kept until ``close``; ``cross_entropy`` says how
    much it takes."""

    # These run on every call: a good tensor takes few attribute reads and no
    # further calls (a small lookup is bound by this code).
    def _matrix(self, t, name, dtypes, rows=None, cols=None):
        """(pointer, row pitch) of a checked matrix."""
        if not isinstance(t, _Tensor) or t.get_device() != self.device or t.dtype not in dtypes:
            self._refuse(t, name, dtypes)
        shape = t.shape
        if len(shape) != 2 or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
            raise ValueError(f"{name} has shape {tuple(shape)}, expected ({'*' if rows is None else rows}, "
                             f"{'*' if cols is None else cols})")
        pitch, step = t.stride()
        if step != 1 and shape[1] > 1:
            raise ValueError(f"{name} must have contiguous rows")
        if shape[0] <= 1:
            pitch = shape[1]
        elif pitch < shape[1]:
            raise ValueError(f"{name} has overlapping rows (stride {pitch})")
        return t.data_ptr(), pitch

    # ----------------------------------------------------------- embedding
    def _embed(self, fn, ids, table, rows, scale, flags, stream):
        table_p, ld_table = self._matrix(table, "table", _FLOATS)
        vocab, dim = table.shape
        n = ids.numel()
        rows_p, ld_rows = self._matrix(rows, "rows", _FLOATS, n, dim)
        self._call(fn, capi.DmuonEmbed(n, vocab, dim, self._list(ids, "ids", _INDEX, n), table_p, rows_p, ld_table,
                                       ld_rows, _INDEX[ids.dtype], _FLOATS[table.dtype], _FLOATS[rows.dtype], scale, flags),
                   stream)

    def embed(self, ids, table, out=None, scale=1.0, stream=None):
        """out[i] = scale * table[ids[i]] (zeros for ids below zero); returns
        ``out`` (allocated on ``stream``, in the table's dtype, if None)."""
        if out is None:
            self._matrix(table, "table", _FLOATS)
            if not isinstance(ids, _Tensor):
                self._refuse(ids, "ids", _INDEX)
            out = self._empty(stream, ids.numel(), table.shape[1], dtype=table.dtype)
        self._embed(self._lib.dmuon_embed_forward, ids, table, out, scale, 0, stream)
        return out

    def embed_grad(self, ids, dout, dtable, scale=1.0, accumulate=False, stream=None):
        """dtable[v] = scale * sum of dout[i] over ids[i] = v, for the whole
        table; with ``accumulate`` added to what ``dtable`` holds."""
        self._embed(self._lib.dmuon_embed_backward, ids, dtable, dout, scale,
                    capi.DMUON_EMBED_ADD if accumulate else 0, stream)
        return dtable

    # ------------------------------------------------------- cross entropy
    def cross_entropy(self, x, w, targets, weights=None, mean=True, logit_scale=1.0, grad_scale=1.0,
                      loss=None, lse=None, total=None, dx=None, dw=None, accumulate_dw=False, stream=None,
                      fine_grads=False):
        """Softmax cross entropy of logits ``logit_scale * x @ w.T`` against
        ``targets`` (below zero: not counted).

        The logits are not stored; with gradients the scratch holds 16 bits of
        each (32 with two halves, below) between the products, for as many tokens
        at a time as fit in 2 GiB (tuning key 14, in MiB).

        Writes whichever outputs are given: ``loss`` and ``lse`` (fp32 per
        token), ``total`` (one fp32: the weighted sum of losses, over the sum
        of weights with ``mean``), and the gradients of ``grad_scale * total``
        in ``dx`` (like x) and ``dw`` (like w; added to with
        ``accumulate_dw``), bf16 or fp32.  With none given, ``loss`` is
        allocated, on ``stream``.  Returns ``loss``.

        The gradients are products of d logits in bf16; up to 128 tokens, and
        with ``fine_grads`` always, a second bf16 holds what the first rounds
        away (twice the work of both products above 128 tokens)."""
        x_p, ld_x = self._matrix(x, "x", _BF16)
        n, dim = x.shape
        w_p, ld_w = self._matrix(w, "w", _BF16, cols=dim)
        vocab = w.shape[0]
        targets_p = self._list(targets, "targets", _INDEX, n)
        weights_p = loss_p = lse_p = total_p = dx_p = dw_p = None
        ld_dx = ld_dw = dx_type = dw_type = 0
        if loss is None and lse is None and total is None and dx is None and dw is None:
            loss = self._empty(stream, n, dtype=torch.float32)
        if weights is not None:
            weights_p = self._list(weights, "weights", _F32, n)
        if loss is not None:
            loss_p = self._list(loss, "loss", _F32, n)
        if lse is not None:
            lse_p = self._list(lse, "lse", _F32, n)
        if total is not None:
            total_p = self._list(total, "total", _F32, 1)
        if dx is not None:
            dx_p, ld_dx = self._matrix(dx, "dx", _FLOATS, n, dim)
            dx_type = _FLOATS[dx.dtype]
        if dw is not None:
            dw_p, ld_dw = self._matrix(dw, "dw", _FLOATS, vocab, dim)
            dw_type = _FLOATS[dw.dtype]
        a = capi.DmuonCe(n, vocab, dim, x_p, w_p, ld_x, ld_w, targets_p, weights_p, loss_p, lse_p, total_p, dx_p, dw_p,
                         ld_dx, ld_dw, capi.DMUON_DTYPE_BF16, capi.DMUON_DTYPE_BF16, _INDEX[targets.dtype], dx_type,
                         dw_type, logit_scale, grad_scale,
                         (capi.DMUON_CE_MEAN if mean else 0) | (capi.DMUON_CE_ADD_DW if accumulate_dw else 0)
                         | (capi.DMUON_CE_FINE_GRADS if fine_grads else 0))
        self._call(self._lib.dmuon_cross_entropy, a, stream)
        return loss

    # ---------------------------------------------------- log probabilities
    def token_logprobs(self, x, w, tokens=None, logit_scale=1.0, logprobs=None, lse=None, entropy=None, top_ids=None,
                       top_logprobs=None, dlogprobs=None, dentropy=None, grad_scale=1.0, dx=None, dw=None,
                       accumulate_dw=False, stream=None, fine_grads=False):
        """Log probabilities of ``tokens`` under the logits ``logit_scale * x @ w.T``
        (``logit_scale``: one over the temperature), the entropies of the
        distributions, their most likely entries, and the gradients.

        Writes whichever outputs are given: ``logprobs``, ``lse`` and
        ``entropy`` (fp32 per token), ``top_ids`` (int32 or int64, tokens x k,
        k up to 32) with ``top_logprobs`` (fp32, the same shape), in falling
        order, equal ones by ascending id.  With none given, ``logprobs`` is
        allocated, on ``stream``.  Returns ``logprobs``.

        ``tokens`` below zero: the row is not scored (outputs 0, alternatives -1,
        no gradient).  None: every row is scored, with no token given.

        With ``dlogprobs`` and ``dentropy`` (fp32 per token, the gradients of a
        loss with respect to both; either may be None) ``dx`` and ``dw`` are
        the loss's gradients times ``grad_scale``, as in ``cross_entropy``."""
        x_p, ld_x = self._matrix(x, "x", _BF16)
        n, dim = x.shape
        w_p, ld_w = self._matrix(w, "w", _BF16, cols=dim)
        vocab = w.shape[0]
        tokens_p = logprobs_p = lse_p = entropy_p = top_p = top_lp_p = dlogprobs_p = dentropy_p = dx_p = dw_p = None
        ld_dx = ld_dw = dx_type = dw_type = token_type = top_type = n_top = 0
        if logprobs is None and lse is None and entropy is None and top_ids is None and dx is None and dw is None:
            logprobs = self._empty(stream, n, dtype=torch.float32)
        if tokens is not None:
            tokens_p = self._list(tokens, "tokens", _INDEX, n)
            token_type = _INDEX[tokens.dtype]
        if logprobs is not None:
            logprobs_p = self._list(logprobs, "logprobs", _F32, n)
        if lse is not None:
            lse_p = self._list(lse, "lse", _F32, n)
        if entropy is not None:
            entropy_p = self._list(entropy, "entropy", _F32, n)
        if top_ids is not None:
            n_top = top_ids.shape[1] if isinstance(top_ids, _Tensor) and top_ids.dim() == 2 else 0
            top_p = self._list(top_ids, "top_ids", _INDEX, n * n_top)
            if top_ids.dim() != 2 or top_ids.shape[0] != n:
                raise ValueError(f"top_ids has shape {tuple(top_ids.shape)}, expected ({n}, *)")
            top_type = _INDEX[top_ids.dtype]
        if top_logprobs is not None:
            if top_ids is None:
                raise ValueError("top_logprobs without top_ids")
            top_lp_p = self._list(top_logprobs, "top_logprobs", _F32, n * n_top)
            if top_logprobs.shape != top_ids.shape:
                raise ValueError(f"top_logprobs has shape {tuple(top_logprobs.shape)}, expected {tuple(top_ids.shape)}")
        if dlogprobs is not None:
            dlogprobs_p = self._list(dlogprobs, "dlogprobs", _F32, n)
        if dentropy is not None:
            dentropy_p = self._list(dentropy, "dentropy", _F32, n)
        if dx is not None:
            dx_p, ld_dx = self._matrix(dx, "dx", _FLOATS, n, dim)
            dx_type = _FLOATS[dx.dtype]
        if dw is not None:
            dw_p, ld_dw = self._matrix(dw, "dw", _FLOATS, vocab, dim)
            dw_type = _FLOATS[dw.dtype]
        a = capi.DmuonLogprobs(n, vocab, dim, x_p, w_p, ld_x, ld_w, tokens_p, logprobs_p, lse_p, entropy_p, top_p, top_lp_p,
                               dlogprobs_p, dentropy_p, dx_p, dw_p, ld_dx, ld_dw, capi.DMUON_DTYPE_BF16,
                               capi.DMUON_DTYPE_BF16, token_type, top_type, dx_type, dw_type, n_top, logit_scale,
                               grad_scale, (capi.DMUON_CE_ADD_DW if accumulate_dw else 0)
                               | (capi.DMUON_CE_FINE_GRADS if fine_grads else 0))
        self._call(self._lib.dmuon_token_logprobs, a, stream)
        return logprobs
