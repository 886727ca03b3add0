"""The paged-cache operators together, as a serving loop uses them: prompts, decoding with
requests that come, grow and end, and the same step captured once and replayed."""
import numpy as np
import pytest
import torch

from tests import test_parity_paged as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from learned_relative_gqa_b200 import build
    build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("window,clip", [(0, False), (48, True)])
def test_prompt_then_decode_is_the_whole_sequence_forward(window, clip):
    """A prompt by the training forward and its keys appended; then each next token decoded
    from the cache equals that row of the forward over the whole sequence. Both are within
    1e-2 (out) and 1e-3 (lse) of the formula by their own parity tests: the sum of the
    forward's 1e-2 / 1e-3 and the decode's, which is far below, bounds the difference."""
    from learned_relative_gqa_b200 import binding
    from learned_relative_gqa_b200.paged import PagedKVCache
    g = P.gen(3)
    B, L, prompt, Hq, Hkv, D, R = 3, 150, [130, 1, 77], 8, 2, 128, 64
    bf = lambda *s, f=1.0: (f * torch.randn(s, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    q, k, v, prof = bf(B, L, Hq, D), bf(B, L, Hkv, D), bf(B, L, Hkv, D), bf(B, Hq, L, R, f=0.5)
    sink = torch.randn(B, L, Hq, generator=g, device="cuda")
    valid = torch.ones(B, L, dtype=torch.bool, device="cuda")
    kw = dict(threshold=9.0, clip_scale=1 + 0.1 * torch.rand(Hkv, D, generator=g, device="cuda")) if clip else {}
    kc = binding.l2clip_forward(k, 9.0, kw["clip_scale"]) if clip else k
    out, lse = binding.forward(q, kc, v, prof, sink, valid, window=window)
    cache = PagedKVCache(max_requests=B, max_len=L, num_pages=32, page_size=16, heads_kv=Hkv, head_dim=D)
    plan = cache.reserve(i32(prompt), 256)
    rows = [(b, i) for b in range(B) for i in range(prompt[b])]
    b, i = torch.tensor(rows, device="cuda").T
    n = len(rows)
    assert torch.equal(plan["positions"][:n].long(), i) and (plan["slots"][n:] == -1).all()
    pad = lambda x: torch.cat([x, torch.full((256 - n, Hkv, D), float("nan"), device="cuda").to(x.dtype)])  # noqa: E731
    cache.append(pad(k[b, i]), pad(v[b, i]), plan["slots"], **kw)
    for step in range(20):
        at = [p + step for p in prompt]
        rows = torch.arange(B, device="cuda")
        plan = cache.reserve(i32([a + 1 for a in at]), B)
        assert plan["positions"].tolist() == at
        now = torch.tensor(at, device="cuda")
        cache.append(k[rows, now], v[rows, now], plan["slots"], **kw)
        o, s = cache.decode(q[rows, now], prof[rows, :, now].contiguous(), sink[rows, now].contiguous(), window=window)
        assert (o - out[rows, now]).abs().max() <= 1.1e-2
        assert (s - lse[rows, now]).abs().max() <= 1.1e-3
    assert cache.info[2] == 0


def test_a_step_on_a_stream_of_its_own():
    """Every call with ``stream=``: the results are those of the current stream."""
    from learned_relative_gqa_b200.paged import PagedKVCache
    g = P.gen(5)
    kw = dict(max_requests=3, max_len=100, num_pages=30, page_size=16, heads_kv=2, head_dim=64)
    k, v = (torch.randn(120, 2, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(3, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
    sink = torch.randn(3, 4, generator=g, device="cuda")
    got = []
    for st in (None, torch.cuda.Stream()):
        cache = PagedKVCache(**kw)
        want, again = i32([50, 0, 70]), i32([0, 33, 72])
        if st is not None:
            st.wait_stream(torch.cuda.current_stream())
        for lens in (want, again):
            plan = cache.reserve(lens, 120, stream=st)
            cache.append(k, v, plan["slots"], stream=st)
            out = cache.decode(q, sink=sink, stream=st)
        if st is not None:
            torch.cuda.current_stream().wait_stream(st)
        got.append([*out, plan["slots"], plan["positions"], cache.lens.clone(), cache.info.clone()])
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("own_stream", [False, True])
def test_entry_points_with_buffers_of_the_caller(own_stream):
    """The C entry points' names on the caller's own buffers: the same bits as the allocating calls."""
    from learned_relative_gqa_b200 import binding as B
    x, s = P.problem([130, 0, 33], 8, 2, 64, 16, 24, "e4m3", "hnd", seed=31, poison=False)
    old, new = i32([130, 0, 33]), i32([150, 12, 0])
    table, num_pages = torch.nn.functional.pad(x["block_table"], (0, 4), value=-1), x["k_cache"].shape[0]
    free = torch.cat([torch.tensor([p for p in range(num_pages) if p not in table.tolist()[0] + table.tolist()[2]],
                                   dtype=torch.int32, device="cuda"), torch.full((num_pages,), -1, dtype=torch.int32,
                                                                                 device="cuda")])[:num_pages].contiguous()
    count = i32([int((free >= 0).sum())])
    g = P.gen(32)
    k, v = (torch.randn(40, 2, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    states = [[t.clone() for t in (table, free, x["k_cache"].contiguous(), x["v_cache"].contiguous())] for _ in range(2)]
    q, prof, sink = x["q"], x["profiles"], x["sink"]
    (t0, f0, kc, vc), (t1, f1, kd, vd) = states
    plan = B.kv_plan(old, new, t0, f0, count, page_size=16, num_pages=num_pages, max_tokens=40)
    B.kv_append(k, v, plan["slots"], kc, vc, **s, threshold=7.0)
    want = B.paged_decode(q, kc, vc, t0, plan["lens"], prof, sink, window=50, **s)
    st = torch.cuda.Stream() if own_stream else None
    lens, start, pos, info = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (3, 4, 40, 4))
    slots = torch.empty(40, dtype=torch.int64, device="cuda")
    out, lse = torch.empty(3, 8, 64, device="cuda"), torch.empty(3, 8, device="cuda")
    desc = B.make_kv_cache_desc(kd, vd)
    dims = B.DecodeDims(3, 8, 24, 50, t1.shape[1], 0.0)
    ws = B.alloc_decode_workspace(desc, dims, "cuda")
    if st is not None:
        st.wait_stream(torch.cuda.current_stream())
    B.inkling_kv_plan(B.KVPlanDims(3, 16, t1.shape[1], num_pages, 40), old, new, t1, f1, count, lens, start, slots, pos,
                      info, st)
    B.inkling_kv_append(desc, B.KVAppendDims(40, 128, 128, 1, 7.0), k, v, slots, s["k_scale"], s["v_scale"], None, None,
                        kd, vd, st)
    B.inkling_rel_attn_decode(desc, dims, q, kd, vd, s["k_scale"], s["v_scale"], prof, sink, t1, lens, out, lse, ws, st)
    if st is not None:
        torch.cuda.current_stream().wait_stream(st)
    for a, b in ((out, want[0]), (lse, want[1]), (t1, t0), (f1, f0), (lens, plan["lens"]), (start, plan["query_start"]),
                 (slots, plan["slots"]), (pos, plan["positions"]), (info, plan["info"]),
                 (kd.view(torch.uint8), kc.view(torch.uint8)), (vd.view(torch.uint8), vc.view(torch.uint8))):
        assert torch.equal(a, b)


def test_wrong_tensors_are_refused():
    from learned_relative_gqa_b200 import binding
    from learned_relative_gqa_b200.paged import PagedKVCache
    cache = PagedKVCache(max_requests=2, max_len=64, num_pages=8, page_size=16, heads_kv=2, head_dim=64)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    prof = torch.zeros(2, 4, 12, dtype=torch.bfloat16, device="cuda")
    for bad, match in ((dict(q=q[:1]), "block_table"), (dict(q=q.float()), "bfloat16|BFloat16"),
                       (dict(q=q.transpose(0, 1)), "contiguous|shape"), (dict(q=q[:, :, :32]), "head_dim"),
                       (dict(q=q.cpu()), "expected cuda"), (dict(sink=torch.zeros(2, 3, device="cuda")), "sink"),
                       (dict(profiles=prof[:, :3].contiguous()), "profiles"),
                       (dict(workspace=torch.zeros(4, device="cuda")), "workspace")):
        with pytest.raises(ValueError, match=match):
            cache.decode(**dict(dict(q=q), **bad))
    with pytest.raises(binding.InklingError, match="unsupported"):
        cache.decode(q, prof)  # an extent that is no multiple of 8
    with pytest.raises(binding.InklingError, match="invalid"):
        cache.decode(q[:, :3].contiguous())  # 3 query heads for 2 KV heads
    with pytest.raises(binding.InklingError, match="invalid"):
        cache.decode(q, window=-1)
    with pytest.raises(binding.InklingError, match="invalid"):
        cache.decode(q, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="dense"):
        cache.append(k.transpose(1, 2).contiguous().transpose(1, 2), k, slots)
    with pytest.raises(ValueError, match="slots"):
        cache.append(k, k, slots.int())
    with pytest.raises(ValueError, match="threshold"):
        cache.append(k, k, slots, tau=torch.ones(3, device="cuda"))
    with pytest.raises(binding.InklingError, match="invalid"):
        cache.append(k, k, slots, threshold=-1.0)
    with pytest.raises(binding.InklingError, match="invalid"):
        cache.append(k[:1].expand(3, 2, 64), k, slots)  # rows on top of each other
    with pytest.raises(binding.InklingError, match="invalid"):
        binding.kv_append(k, k, slots, cache.k_cache, cache.k_cache)
    lens = i32([1, 2])
    with pytest.raises(ValueError, match="new_lens"):
        cache.reserve(i32([1, 2, 3]), 4)
    with pytest.raises(binding.InklingError, match="invalid"):  # an output over an input
        binding.kv_plan(cache.lens, lens, cache.block_table, cache.free_pages, cache.info[:1], page_size=16,
                        num_pages=8, max_tokens=4, lens=lens)
    assert not cache.lens.any() and int(cache.info[0]) == 8


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_captured_step_serves_requests_that_come_and_go(dtype):
    """One graph of plan, append and decode, replayed with new lengths: pages move between
    requests, and every row is the oracle's over what was appended for it."""
    from learned_relative_gqa_b200.paged import PagedKVCache
    g = P.gen(4)
    N, Hq, Hkv, D, R, page, num_pages = 6, 8, 2, 64, 32, 4, 40
    scale = {} if dtype == "bf16" else dict(dtype=torch.float8_e4m3fn, k_scale=torch.full((Hkv,), 0.011, device="cuda"),
                                            v_scale=torch.full((Hkv,), 0.013, device="cuda"))
    cache = PagedKVCache(max_requests=N, max_len=64, num_pages=num_pages, page_size=page, heads_kv=Hkv, head_dim=D,
                         **scale)
    T = 64
    k, v = (torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(N, Hq, D, dtype=torch.bfloat16, device="cuda")
    prof = torch.zeros(N, Hq, R, dtype=torch.bfloat16, device="cuda")
    sink = torch.zeros(N, Hq, device="cuda")
    want = i32([0] * N)
    state = (cache.block_table, cache.free_pages, cache._state)
    saved = [t.clone() for t in state]

    def step():
        plan = cache.reserve(want, T)
        cache.append(k, v, plan["slots"])
        return plan, cache.decode(q, prof, sink)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, (out, lse) = step()
    for t, s in zip(state, saved):
        t.copy_(s)
    rng = np.random.default_rng(8)
    lens = [0] * N
    for turn in range(12):
        new = []
        for x in lens:
            if x == 0:
                new.append(int(rng.integers(0, 20)))
            else:
                new.append(0 if rng.random() < 0.3 else min(64, x + int(rng.integers(0, 4))))
        if turn == 11:
            new = [64] * N  # more than the pool holds: 40 pages of 4 for 6 x 64 tokens
        for t in (k, v, q, prof):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        sink.copy_(torch.randn(sink.shape, generator=g, device="cuda"))
        want.copy_(i32(new))
        graph.replay()
        torch.cuda.synchronize()
        granted = cache.lens.tolist()
        if turn < 11:
            assert granted == new and cache.info[2] == 0
        else:
            assert cache.info[2] > 0 and cache.info[0] == 0 and sum(-(-x // page) for x in granted) == num_pages
        # no page is in two tables, or in a table and free
        held = [p for n, x in enumerate(granted) for p in cache.block_table[n, :-(-x // page)].tolist()]
        free = cache.free_pages[:int(cache.info[0])].tolist()
        assert sorted(held + free) == list(range(num_pages))
        # the new rows are where the table says
        start = plan["query_start"].tolist()
        for n in range(N):
            for i in range(lens[n], granted[n]):
                t = start[n] + i - lens[n]
                if t >= T:
                    continue
                got = cache.k_cache[cache.block_table[n, i // page].long(), i % page]
                if dtype == "bf16":
                    assert torch.equal(got, k[t])
                else:
                    y = (k[t].float() / 0.011).clamp(-448, 448).to(torch.float8_e4m3fn)
                    assert torch.equal(got.view(torch.uint8), y.view(torch.uint8))
        x = dict(q=q, k_cache=cache.k_cache, v_cache=cache.v_cache, block_table=cache.block_table, lens=cache.lens,
                 profiles=prof, sink=sink)
        P.check(x, dict(k_scale=cache.k_scale, v_scale=cache.v_scale), got=(out, lse))
        lens = granted
