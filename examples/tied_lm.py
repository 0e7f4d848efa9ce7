"""A small language model trained with everything the package offers a step:
embedding lookup, cross entropy over the tied head, their gradients, and the
owner step (Muon for the matrices, AdamW for the table).

    x = T[id] + relu(T[id] A) B        logits = x T^T        (T tied)

T's gradient has two parts: the head's (cross entropy, written) and the
lookup's (added to it).  The hidden layer is plain torch.  The data is a random
Markov chain whose entropy is known, so the loss has a floor to compare with.

    python examples/tied_lm.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import matrix_optimizer_step_gb300 as mos  # noqa: E402


def chain(vocab, n_next, generator):
    """A Markov chain: each id is followed by one of n_next ids, evenly."""
    return torch.randint(0, vocab, (vocab, n_next), generator=generator, device="cuda")


def draw(table, batch, length, generator):
    ids = torch.empty(batch, length + 1, dtype=torch.int64, device="cuda")
    ids[:, 0] = torch.randint(0, table.shape[0], (batch,), generator=generator, device="cuda")
    for i in range(length):
        pick = torch.randint(0, table.shape[1], (batch,), generator=generator, device="cuda")
        ids[:, i + 1] = table[ids[:, i], pick]
    return ids


class TiedLM:
    def __init__(self, vocab=5003, dim=256, hidden=512, tokens=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        shapes = {"table": (vocab, dim), "A": (dim, hidden), "B": (hidden, dim)}
        std = {"table": dim ** -0.5, "A": dim ** -0.5, "B": hidden ** -0.5}
        self.master = {k: torch.randn(s, generator=g, device="cuda") * std[k] for k, s in shapes.items()}
        self.param = {k: v.to(torch.bfloat16) for k, v in self.master.items()}
        # The table's gradient is a sum of two operators' results: fp32 keeps it to one rounding each.
        self.grad = {k: torch.zeros(s, device="cuda", dtype=torch.float32 if k == "table" else torch.bfloat16)
                     for k, s in shapes.items()}
        state = {k: [torch.zeros_like(v) for _ in range(2)] for k, v in self.master.items()}
        self.ops, self.owner = mos.VocabOps(0), mos.OwnerStep(0)
        mats = ("A", "B")
        self.owner.set_muon([self.master[k] for k in mats], [state[k][0] for k in mats], [self.grad[k] for k in mats],
                            [self.param[k] for k in mats])
        self.owner.set_adamw([self.master["table"]], [state["table"][0]], [state["table"][1]], [self.grad["table"]],
                             [self.param["table"]])
        self.h = torch.empty(tokens, dim, device="cuda", dtype=torch.bfloat16)
        self.dx = torch.empty_like(self.h)
        self.total = torch.zeros(1, device="cuda")
        self.steps = 0

    def gradients(self, ids, targets):
        """Forward and backward of one batch: fills self.grad, returns the mean loss (on the device)."""
        T, A, B = self.param["table"], self.param["A"], self.param["B"]
        h = self.ops.embed(ids, T, self.h)
        a = h @ A
        r = torch.relu(a)
        x = h + r @ B
        # Loss, its gradient with respect to x, and the head's part of the table's gradient.
        self.ops.cross_entropy(x, T, targets, total=self.total, dx=self.dx, dw=self.grad["table"])
        self.grad["B"].copy_(r.T @ self.dx)
        da = (self.dx @ B.T) * (a > 0)
        self.grad["A"].copy_(h.T @ da)
        dh = self.dx + da @ A.T
        # The lookup's part is added.
        self.ops.embed_grad(ids, dh, self.grad["table"], accumulate=True)
        return self.total

    def step(self, ids, targets, lr=0.02, adam_lr=3e-3):
        loss = self.gradients(ids, targets)
        self.steps += 1
        self.owner.step(dict(lr=lr, momentum=0.95, wd=0.0),
                        dict(lr=adam_lr, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.0, step=self.steps))
        return loss

    def sync(self):
        self.ops.sync()
        self.owner.sync()


def main(steps=300, batch=64, length=64, n_next=4):
    g = torch.Generator(device="cuda").manual_seed(1)
    model = TiedLM(tokens=batch * length)
    table = chain(model.param["table"].shape[0], n_next, g)
    losses = []
    for i in range(steps):
        ids = draw(table, batch, length, g)
        loss = model.step(ids[:, :-1].reshape(-1), ids[:, 1:].reshape(-1))
        if i % max(1, steps // 10) == 0 or i == steps - 1:
            model.sync()
            losses.append(float(loss))
            print(f"step {i:4d}  loss {losses[-1]:.4f}  (the chain's entropy: {torch.log(torch.tensor(float(n_next))):.4f})")
    return losses


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
