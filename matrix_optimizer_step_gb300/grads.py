"""User-facing wrapper of the gradient operators: norms of many tensors, and
clipping to a global norm.

``GradOps`` keeps a library context; a list of gradients is registered once and
then handed to its methods, so a training loop does not marshal pointers every
step.  ``OwnerStep.step(..., max_norm=)`` clips the owner's own gradients without
writing them.
"""

from __future__ import annotations

import torch

from . import capi
from .vocab import _F32, _FLOATS, Ops


class GradList:
    """Registered gradients (``GradOps.register``); keeps the tensors."""

    def __init__(self, array, n, tensors, outs):
        self.array, self.n, self.tensors, self.outs = array, n, tensors, outs

    def __len__(self):
        return self.n


class GradOps(Ops):
    """Gradient norms and clipping on one GPU.

    Gradients are bf16 or fp32 tensors of any shape, contiguous.  Work is
    enqueued on ``stream`` (a torch stream or handle; None: the current one) and
    returns without waiting, and no value comes to the host; ``sync`` waits.  The
    handle's scratch comes from CUDA and is kept until ``close``."""

    def register(self, grads, outs=None):
        """A list of gradients for the methods below, and where ``clip`` and
        ``scale`` write (bf16 or fp32 tensors of the same sizes; None: in place)."""
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if len(outs) != len(grads):
            raise ValueError("one out per gradient")
        descs = (capi.DmuonGrad * max(len(grads), 1))()
        for i, (g, o) in enumerate(zip(grads, outs)):
            for t, name in ((g, f"grads[{i}]"), (o, f"outs[{i}]")):
                if not isinstance(t, torch.Tensor) or t.get_device() != self.device or t.dtype not in _FLOATS:
                    self._refuse(t, name, _FLOATS)
                if t.numel() != g.numel() or not t.is_contiguous():
                    raise ValueError(f"{name}: expected {g.numel()} contiguous elements")
            descs[i] = capi.DmuonGrad(g.numel(), g.data_ptr(), o.data_ptr(), _FLOATS[g.dtype], _FLOATS[o.dtype])
        return GradList(descs, len(grads), grads, outs)

    def _listed(self, grads):
        return grads if isinstance(grads, GradList) else self.register(grads)

    def _result(self, t, name, n):
        return None if t is None else self._list(t, name, _F32, n)

    def norm(self, grads, norm=None, norms=None, coef=None, max_norm=None, stream=None):
        """2-norm of all ``grads`` (a registered list or tensors) together into
        ``norm``, of each into ``norms`` and, with ``max_norm``,
        min(1, max_norm / (norm + 1e-6)) into ``coef``: fp32 tensors on the
        device, whichever are given; with none, ``norm`` is allocated.
        Returns ``norm``."""
        grads = self._listed(grads)
        if norm is None and norms is None and coef is None:
            norm = self._empty(stream, 1, dtype=torch.float32)
        if coef is not None and max_norm is None:
            raise ValueError("coef needs max_norm")
        capi._check(self._lib.dmuon_grad_norm(
            self.ctx, grads.array, grads.n, 0.0 if max_norm is None else float(max_norm), self._result(norm, "norm", 1),
            self._result(norms, "norms", grads.n), self._result(coef, "coef", 1), self._stream(stream)))
        return norm

    def clip(self, grads, max_norm, norm=None, norms=None, coef=None, stream=None):
        """Every gradient times min(1, max_norm / (norm + 1e-6)), in place or into
        the registered outs; results as in ``norm``.  Returns ``norm``."""
        grads = self._listed(grads)
        if norm is None:
            norm = self._empty(stream, 1, dtype=torch.float32)
        capi._check(self._lib.dmuon_clip_grads(
            self.ctx, grads.array, grads.n, float(max_norm), self._result(norm, "norm", 1),
            self._result(norms, "norms", grads.n), self._result(coef, "coef", 1), self._stream(stream)))
        return norm

    def scale(self, grads, coef, stream=None):
        """Every gradient times ``coef`` (one fp32 on the device), in place or into the registered outs."""
        grads = self._listed(grads)
        capi._check(self._lib.dmuon_scale_grads(self.ctx, grads.array, grads.n, self._list(coef, "coef", _F32, 1),
                                                self._stream(stream)))
