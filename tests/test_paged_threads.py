"""Serving steps of two host threads at once, each with a cache and a stream of its own: the bits of either
alone."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from learned_relative_gqa_b200 import build
    build.build()


def serve(kind, results, start=None):
    """Steps of one cache on a stream of its own; the results of every step, on the host."""
    from learned_relative_gqa_b200.paged import PagedKVCache
    try:
        e4m3 = kind % 2 == 1
        g = torch.Generator("cuda").manual_seed(kind)
        N, hkv, D, hq = (5, 2, 64, 8) if e4m3 else (9, 1, 128, 12)
        scales = dict(dtype=torch.float8_e4m3fn, k_scale=torch.full((hkv,), 0.011, device="cuda"),
                      v_scale=torch.full((hkv,), 0.013, device="cuda")) if e4m3 else {}
        st = torch.cuda.Stream()
        rng = np.random.default_rng(kind)
        got = []
        with torch.cuda.stream(st):
            cache = PagedKVCache(max_requests=N, max_len=3000, num_pages=N * 200, page_size=16, heads_kv=hkv,
                                 head_dim=D, **scales)
            lens = np.zeros(N, dtype=np.int64)
            st.synchronize()
            if start is not None:
                start.wait(60)
            for step in range(12):
                lens = np.where(rng.random(N) < 0.2, 0, np.minimum(3000, lens + rng.integers(1, 400 if step < 6 else 2, N)))
                plan = cache.reserve(torch.tensor(lens, dtype=torch.int32).cuda(), N * 400)
                k, v = (torch.randn(N * 400, hkv, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
                cache.append(k, v, plan["slots"], threshold=9.0)
                q = torch.randn(N, hq, D, generator=g, device="cuda").to(torch.bfloat16)
                prof = torch.randn(N, hq, 64, generator=g, device="cuda").to(torch.bfloat16)
                for window in (0, 200):
                    got += cache.decode(q, prof, window=window)
                got += [plan["slots"], plan["positions"], cache.lens.clone(), cache.info.clone()]
            st.synchronize()
            results[kind] = [t.cpu() for t in got]
    except Exception as e:  # noqa: BLE001
        results[kind] = repr(e)


def test_two_threads_serve_side_by_side():
    alone, together = {}, {}
    for kind in (0, 1):
        serve(kind, alone)
    start = threading.Barrier(2)
    threads = [threading.Thread(target=serve, args=(kind, together, start)) for kind in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for kind in (0, 1):
        assert not isinstance(alone[kind], str) and not isinstance(together[kind], str), (alone[kind], together[kind])
        assert all(torch.equal(a, b) for a, b in zip(alone[kind], together[kind]))
        assert all(torch.isfinite(t).all() or i % 8 in (1, 3) for i, t in enumerate(alone[kind]))
