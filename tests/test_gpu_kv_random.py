"""Attention over the 8-bit cache on calls drawn at random: how many tokens sequences bring, their lengths, heads,
masks, scales, types, with offsets or without, bounds or none, whole items or runs on few or many SMs."""
from __future__ import annotations

import random

import pytest
import torch

from tests import kv_util as U
from tests.kv_check import check
from tests.test_gpu_kv import gdn  # noqa: F401

pytestmark = pytest.mark.gpu


def draw(r: random.Random):
    h_kv = r.choice([1, 2, 3, 4])
    h_q = r.choice([h_kv, 2 * h_kv, 4 * h_kv, h_kv + 1, 5 * h_kv])
    n = r.choice([1, 1, 2, 3, 5, 9, 40, 150, 300])
    most = 10 if n >= 40 else 200
    tokens = {"decode": lambda: 1, "few": lambda: r.randint(0, 9), "many": lambda: r.randint(1, most),
              "mixed": lambda: r.choice([0, 1, 1, 2, 5, r.randint(1, most)])}[r.choice(["decode", "few", "many", "mixed"])]
    q = [tokens() for _ in range(n)]
    if sum(q) == 0 or r.random() < 0.3:
        q = [max(1, q[0])] * n
    past = lambda x: r.choice([0, -1, -3, r.randint(0, 70), r.randint(0, 900 if n < 40 else 200), 64 - x, 128])  # noqa: E731
    return q, [max(0, x + past(x)) for x in q], h_q, h_kv


@pytest.mark.parametrize("seed", range(60))
def test_attn(gdn, seed):  # noqa: F811
    r = random.Random(seed)
    q_lens, kv_lens, h_q, h_kv = draw(r)
    dtype = r.choice([torch.bfloat16, torch.bfloat16, torch.float32])
    b = U.Batch(q_lens, kv_lens, h_kv, seed=seed, spread=r.choice([0.2, 1.0, 2.0]))
    b.fill()
    q = b.randn(b.T, h_q, 128) * r.choice([1.0, 0.01, 5.0])
    if r.random() < 0.2:
        q[r.randrange(b.T)] = 0.0
    longest = r.choice([0, max(kv_lens), 20000, 64])
    plan = gdn.gdn_kv_attn_plan(T=b.T, n_seqs=b.n, h_q=h_q, h_kv=h_kv, max_q_len=r.choice([0, max(q_lens)]), max_kv_len=longest,
                                max_pages=max(b.max_pages, -(-longest // 64)), dtype=dtype, causal=r.random() < 0.75,
                                window=r.choice([0, 0, 1, r.randint(1, 300)]), scale=r.choice([0.0, 0.0, 0.1, -0.05, 0.5]),
                                sm_count=r.choice([152, 1, 3, 8, 40]))
    check(gdn, b, h_q, plan, q=q, use_cu=len(set(q_lens)) > 1 or r.random() < 0.5, dtype=dtype)
