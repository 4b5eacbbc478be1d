"""The hybrid-stack example: prefill then captured decode steps give what one longer prefill gives."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("lens,steps", [([130, 1, 64, 63], 5), ([700], 3), ([5] * 9, 70)])
def test_steps_continue_the_prefill(ex, lens, steps):
    """Each step's output against the same token's in a prefill of the whole
    sequence.  The paths round differently (chunked fp16 products against fp32
    steps; a page's scale may still grow, which only moves subnormal codes), by
    the 2e-2 RMS bar of the bf16 paths a mixer; eight residual layers of
    comparable size add up to less than 5 of them."""
    width, batch = 256, len(lens)
    gen = torch.Generator("cuda").manual_seed(3)
    seqs = [torch.randn(n + steps, width, device="cuda", generator=gen).bfloat16() for n in lens]
    whole = ex.HybridStack(width=width, batch=batch, max_tokens=1024).prefill(torch.cat(seqs), [n + steps for n in lens])
    stack = ex.HybridStack(width=width, batch=batch, max_tokens=1024)
    first = stack.prefill(torch.cat([s[:n] for s, n in zip(seqs, lens)]), lens)
    at = torch.tensor([0] + [n + steps for n in lens]).cumsum(0).tolist()
    rms = whole.float().pow(2).mean().sqrt().item()
    begin = torch.cat([whole[a:a + n] for a, n in zip(at, lens)])
    assert (first.float() - begin.float()).abs().max().item() <= 0.1 * rms
    for t in range(steps):
        y = stack.step(torch.stack([s[n + t] for s, n in zip(seqs, lens)]))
        want = torch.stack([whole[a + n + t] for a, n in zip(at, lens)])
        assert (y.float() - want.float()).abs().max().item() <= 0.1 * rms
    assert stack.kv_lens.tolist() == [n + steps for n in lens]


def test_example_runs(ex, capsys):
    ex.main()
    assert "lengths [720, 84, 21, 1310]" in capsys.readouterr().out


def test_prompts_after_the_step_was_captured(ex):
    """New prompts on a stack whose step has been captured: its steps go on from them, as a new stack's do."""
    width, lens = 256, [70, 3, 128]
    gen = torch.Generator("cuda").manual_seed(5)
    rand = lambda n: torch.randn(n, width, device="cuda", generator=gen).bfloat16()  # noqa: E731
    used, new = (ex.HybridStack(width=width, batch=3, max_tokens=512) for _ in range(2))
    used.prefill(rand(40), [9, 30, 1])
    for _ in range(2):
        used.step(rand(3))
    x, tokens = rand(sum(lens)), [rand(3) for _ in range(3)]
    assert torch.equal(used.prefill(x, lens), new.prefill(x, lens))
    for t in tokens:
        assert torch.equal(used.step(t), new.step(t))
