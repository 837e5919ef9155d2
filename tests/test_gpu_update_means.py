"""A gradient that is rounded at random on its way to the optimizer, and the
optimizer's 8-bit average that is rounded at random after it: the mean over many
values is the gradient's, which it is only if two different numbers decide."""
import importlib.util
import inspect
import os
from types import SimpleNamespace

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
N = 1 << 18


@pytest.fixture(scope="module")
def gq():
    from communication_efficient_gradient_amd import gq
    return gq


def example():
    spec = importlib.util.spec_from_file_location(
        "experts_step", os.path.join(ROOT, "examples", "experts_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def gradient():
    """The largest of each bucket of 512 is 1, the others lie in the middle of
    two of INT8's levels, 63 / 127 and 64 / 127."""
    g = torch.full((N,), 0.5, device="cuda")
    g[::512] = 1.0
    return g


def check(m):
    """0.1 of 63 / 127 and of 64 / 127 lie between the codes 12 and 13 times 2^-8:
    a value's rounding is off by at most 2^-8 either way, so by a standard
    deviation of half of that at most, and the gradient's by half of 0.1 / 127."""
    got = m[0].float() * m[1].repeat_interleave(256)
    got = got.view(-1, 512)[:, 1:].double()
    assert set(got.unique().tolist()) <= {12 * 2.0 ** -8, 13 * 2.0 ** -8}
    spread = (0.5 * 2.0 ** -8 + 0.5 * 0.1 / 127) / got.numel() ** 0.5
    assert abs(float(got.mean()) - 0.05) < 5 * spread


@pytest.mark.gpu
def test_the_example_keeps_the_mean(gq):
    b = SimpleNamespace(flat=torch.zeros(N, device="cuda"), grad=gradient(),
                        norm=torch.empty(1, device="cuda"), scale=torch.empty(1, device="cuda"),
                        ws=gq.alloc_workspace(gq.gq_grad_norm_workspace(N)),
                        layers=torch.tensor([0, N], device="cuda"),
                        decay=torch.zeros(1, device="cuda"), pack_weights=lambda: None)
    tr = example().Trainer(b, lr=1e-3, max_norm=float("inf"))
    tr.update()
    check(tr.m)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [0, 1, 7, 1 << 40])
def test_an_update_without_a_seed_keeps_the_mean(gq, seed):
    d, a = gq.desc(gq.GQ_UNIFORM, bucket=512, s=127), gq.adamw(1e-3, bits=8)
    codes, meta = gq.alloc_payload(d, N)
    p, mean = torch.zeros(N, device="cuda"), torch.empty(N, device="cuda")
    m, v = gq.alloc_adamw(a, N)
    gq.gq_quantize(d, gradient(), None, seed, 1, codes, meta)
    gq.gq_dequantize_accumulate(d, N, [codes], [meta], 1.0, 0.0, mean)
    gq.gq_adamw(a, mean, p, m, v, 1)
    check(m)


def test_the_update_has_a_key_of_its_own(gq):
    """No number that a program would think of for its workers."""
    seed = inspect.signature(gq.gq_adamw).parameters["seed"].default
    assert seed == gq.ADAMW_SEED and 1 << 32 < seed < 1 << 64
    mod = example()
    assert mod.Trainer.SEND_SEED != mod.Trainer.UPDATE_SEED
