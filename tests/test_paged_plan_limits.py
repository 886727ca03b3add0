"""The page plan at the sizes where its shared memory passes what a launch gets without asking, and
called by several host threads at once."""
import ctypes
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


def test_plans_of_different_sizes_in_one_graph():
    from learned_relative_gqa_b200 import binding
    cases = [step(N) for N in (16384, 5000, 64)]
    saved = [(x["block_table"].clone(), x["free_pages"].clone()) for x, _, _ in cases]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [binding.kv_plan(**x, **kw) for x, kw, _ in cases]
    for _ in range(2):
        for (x, _, _), (table, free) in zip(cases, saved):
            x["block_table"].copy_(table)
            x["free_pages"].copy_(free)
        graph.replay()
        for g, (x, _, want) in zip(got, cases):
            same(g, x, want)


def test_plans_of_different_sizes_from_two_threads():
    """Two host threads with a stream and buffers each, one with the largest batch and one with a smaller:
    neither may take the other's shared-memory limit away."""
    from learned_relative_gqa_b200 import binding as B
    fails, ready = [], threading.Barrier(2)

    def work(N):
        try:
            x, kw, want = step(N)
            T, M = kw["max_tokens"], x["block_table"].shape[1]
            i32 = dict(dtype=torch.int32, device="cuda")
            out = dict(lens=torch.empty(N, **i32), query_start=torch.empty(N + 1, **i32),
                       slots=torch.empty(T, dtype=torch.int64, device="cuda"), positions=torch.empty(T, **i32),
                       info=torch.empty(4, **i32))
            dims = B.KVPlanDims(N, kw["page_size"], M, kw["num_pages"], T)
            st = torch.cuda.Stream()
            first = {n: x[n].clone() for n in ("block_table", "free_pages")}
            st.wait_stream(torch.cuda.current_stream())
            ready.wait(60)
            # with its arguments made once, so that the threads are inside the library most of the time
            # (repeated plans write the same entries)
            ptr = [ctypes.c_void_p(t.data_ptr()) for t in (*x.values(), *out.values())]
            call, args = B.load().inkling_kv_plan, (ctypes.byref(dims), *ptr, ctypes.c_void_p(st.cuda_stream))
            for _ in range(20000):
                status = call(*args)
                if status != B.INKLING_OK:
                    raise B.InklingError(status, "inkling_kv_plan")
            st.synchronize()
            with torch.cuda.stream(st):
                for n, t in first.items():
                    x[n].copy_(t)
                B.inkling_kv_plan(dims, *x.values(), *out.values(), st)
                st.synchronize()
                same(out, x, want)
        except Exception as e:  # noqa: BLE001
            fails.append((N, repr(e)))

    threads = [threading.Thread(target=work, args=(N,)) for N in (16384, 5000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not fails, fails


def test_plan_with_few_requests_that_give_back_many_pages():
    """Far more pages move than there are requests and tokens: eight requests of 32768 pages end, one that
    grows takes some of those, and the free list was not empty."""
    from learned_relative_gqa_b200 import binding
    N, M, page = 9, 32768, 1
    rng = np.random.default_rng(7)
    old, new = [M] * 8 + [5], [0, M // 2] * 4 + [1005]
    num_pages = 8 * M + 100
    order = rng.permutation(num_pages)
    table = np.full((N, M), -1)
    table[:8], table[8, :5] = order[:8 * M].reshape(8, M), order[8 * M:8 * M + 5]
    free = np.full(num_pages, -1)
    free[:60] = order[8 * M + 5:8 * M + 65]
    want = ref.plan(old, new, table, free, 60, page, 1003, num_pages)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = dict(old_lens=torch.tensor(old, **i32), new_lens=torch.tensor(new, **i32), block_table=torch.tensor(table, **i32),
             free_pages=torch.tensor(free, **i32), free_count=torch.tensor([60], **i32))
    same(binding.kv_plan(**x, page_size=page, num_pages=num_pages, max_tokens=1003), x, want)
