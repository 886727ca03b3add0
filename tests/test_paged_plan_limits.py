"""The page plan at the sizes where its shared memory passes what a launch gets without asking, and
called by several host threads at once."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import paged as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from learned_relative_gqa_b200 import build
    build.build()


def step(N, seed=0):
    """Tables of a step in which every request grows by 0 to 3 tokens, and the oracle's plan of it."""
    rng = np.random.default_rng(seed + N)
    page, M = 4, 3
    old = rng.integers(0, 9, N)
    new = old + rng.integers(0, 4, N)
    held = -(-old // page)
    num_pages = int(held.sum()) + N
    order = rng.permutation(num_pages)
    table, at = np.full((N, M), -1), 0
    for r in range(N):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    free = np.full(num_pages, -1)
    free[:num_pages - at] = order[at:]
    T = int((new - old).sum()) + 5
    want = ref.plan(old, new, table, free, num_pages - at, page, T, num_pages)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = dict(old_lens=torch.tensor(old, **i32), new_lens=torch.tensor(new, **i32), block_table=torch.tensor(table, **i32),
             free_pages=torch.tensor(free, **i32), free_count=torch.tensor([num_pages - at], **i32))
    return x, dict(page_size=page, num_pages=num_pages, max_tokens=T), want


def same(got, x, want):
    got = dict(got, block_table=x["block_table"], free_pages=x["free_pages"])
    for name in want:
        assert np.array_equal(got[name].cpu().numpy(), want[name]), name


def plans(sizes):
    from learned_relative_gqa_b200 import binding
    for N in sizes:
        x, kw, want = step(N)
        same(binding.kv_plan(**x, **kw), x, want)


@pytest.mark.parametrize("sizes", [(4063, 4064, 4095, 4096, 16384), (16384, 4096, 4095, 4064, 1)])
def test_plan_at_the_limit_of_a_launch(sizes):
    """Each order in a process of its own: the first plans of a process may not depend on larger ones before them."""
    code = f"import sys; sys.path.insert(0, {ROOT!r}); from tests import test_paged_plan_limits as t; t.plans({sizes!r})"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
