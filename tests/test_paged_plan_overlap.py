"""CPU-only: the page plan refuses buffers that it would write while it reads or writes them elsewhere."""
import ctypes

import pytest

NAMES = ("old_lens", "new_lens", "block_table", "free_pages", "free_count", "lens", "query_start", "slots", "positions",
         "info")
READ = ("old_lens", "new_lens", "free_count")
N, M, PAGES, T = 4, 10, 50, 100
BYTES = dict(old_lens=4 * N, new_lens=4 * N, block_table=4 * N * M, free_pages=4 * PAGES, free_count=4, lens=4 * N,
             query_start=4 * (N + 1), slots=8 * T, positions=4 * T, info=16)


@pytest.fixture(scope="module")
def lib():
    from learned_relative_gqa_b200 import build, binding
    build.build()
    return binding.load()


def call(lib, **at):
    from learned_relative_gqa_b200.binding import KVPlanDims
    a = {n: 0x1000000 * (i + 1) for i, n in enumerate(NAMES)}
    a.update(at)
    return lib.inkling_kv_plan(ctypes.byref(KVPlanDims(N, 16, M, PAGES, T)), *(ctypes.c_void_p(a[n]) for n in NAMES), None)


@pytest.mark.parametrize("a,b", [(a, b) for i, a in enumerate(NAMES) for b in NAMES[i + 1:]
                                 if not (a in READ and b in READ)])
def test_overlapping_buffers_are_refused(lib, a, b):
    """The same place, and with only the ends on each other."""
    base = 0x1000000 * (NAMES.index(b) + 1)
    assert call(lib, **{a: base}) == 1
    assert call(lib, **{a: base + (BYTES[b] - 4) // 8 * 8}) == 1
    assert call(lib, **{a: base - (BYTES[a] - 4) // 8 * 8}) == 1
