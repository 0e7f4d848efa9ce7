"""The first step of an OwnerStep on a side stream, with the default stream busy: its tables have to be there."""

import pytest
import torch

pytestmark = pytest.mark.gpu

SHAPES = [(256, 512), (384, 128), (1024, 1024), (64, 2048)]


def tensors(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    master = [torch.randn(s, generator=g, device="cuda") for s in SHAPES]
    return dict(master=master, grad=[torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in SHAPES],
                m=[torch.zeros_like(q) for q in master], v=[torch.zeros_like(q) for q in master],
                param=[q.to(torch.bfloat16) for q in master])


def step(mos, stream, busy):
    mats, vecs = tensors(1), tensors(2)
    owner = mos.OwnerStep(0)
    owner.set_muon(mats["master"], mats["m"], mats["grad"], mats["param"])
    owner.set_adamw(vecs["master"], vecs["m"], vecs["v"], vecs["grad"], vecs["param"])
    torch.cuda.synchronize()
    if busy:
        torch.cuda._sleep(int(1.0e8))  # on the default stream
    owner.step(dict(lr=0.02, momentum=0.95, wd=0.0), dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, wd=0.0, step=1),
               stream=stream)
    owner.sync(stream)
    torch.cuda.synchronize()
    return mats["master"] + mats["param"] + vecs["master"] + vecs["param"]


def test_first_step_on_a_side_stream(cuda_lib):
    want = step(cuda_lib, torch.cuda.default_stream(), False)
    for busy in (True, False):
        got = step(cuda_lib, torch.cuda.Stream(), busy)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
