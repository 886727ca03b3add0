"""CPU-only checks of the paged-cache entry points: what they refuse, before anything is launched."""
import ctypes

import pytest
import torch

FAKE, MIS = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    from learned_relative_gqa_b200 import build, binding
    build.build()
    return binding.load()


def cache(**kw):
    from learned_relative_gqa_b200.binding import KVCacheDesc
    d = dict(num_pages=100, page_size=16, heads_kv=4, head_dim=128, dtype=0, page_stride=16 * 4 * 128,
             token_stride=4 * 128, head_stride=128)
    d.update(kw)
    return KVCacheDesc(**d)


def dec(**kw):
    from learned_relative_gqa_b200.binding import DecodeDims
    d = dict(requests=3, heads_q=8, rel_extent=64, window=0, max_pages=10, scale=0.0)
    d.update(kw)
    return DecodeDims(**d)


BAD_CACHE = [(dict(num_pages=0), 1), (dict(page_size=0), 1), (dict(heads_kv=0), 1), (dict(dtype=2), 1),
             (dict(head_dim=96), 2), (dict(num_pages=1 << 31), 2), (dict(page_size=1 << 30), 2),
             (dict(num_pages=1 << 20, page_size=(1 << 11) + 1), 2), (dict(head_stride=64), 1), (dict(token_stride=100), 1),
             (dict(page_stride=-512), 1), (dict(page_stride=0), 1), (dict(head_stride=132), 1),
             (dict(dtype=1, head_stride=136), 1), (dict(page_stride=1 << 58), 2)]


@pytest.mark.parametrize("bad,expect", BAD_CACHE)
def test_cache_descriptor(lib, bad, expect):
    from learned_relative_gqa_b200.binding import KVAppendDims
    c, d, a = cache(**bad), dec(), KVAppendDims(5, 512, 512, 0, 0.0)
    assert lib.inkling_rel_attn_decode_workspace_size(ctypes.byref(c), ctypes.byref(d)) == 0
    assert lib.inkling_rel_attn_decode(ctypes.byref(c), ctypes.byref(d), *([FAKE] * 11), FAKE, 1 << 30, None) == expect
    assert lib.inkling_kv_append(ctypes.byref(c), ctypes.byref(a), FAKE, FAKE, FAKE, None, None, None, None, FAKE,
                                 FAKE, None) == expect


def test_strides_of_single_extents_are_not_looked_at(lib):
    c = cache(num_pages=1, page_size=1, heads_kv=1, page_stride=-7, token_stride=3, head_stride=0)
    assert lib.inkling_rel_attn_decode_workspace_size(ctypes.byref(c), ctypes.byref(dec())) > 0


@pytest.mark.parametrize("bad,expect", [
    (dict(requests=-1), 1), (dict(heads_q=0), 1), (dict(heads_q=6), 1), (dict(rel_extent=-8), 1), (dict(window=-1), 1),
    (dict(max_pages=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(requests=1 << 24), 2),
    (dict(heads_q=65536), 2), (dict(rel_extent=1 << 30), 2), (dict(rel_extent=12), 2), (dict(window=1 << 30), 2), (dict(max_pages=1 << 26), 2),
    (dict(requests=1 << 23, max_pages=1 << 24), 2)])
def test_decode_sizes(lib, bad, expect):
    d = dec(**bad)
    assert lib.inkling_rel_attn_decode_workspace_size(ctypes.byref(cache()), ctypes.byref(d)) == 0
    a = [FAKE] * 11
    a[3] = a[4] = None
    assert lib.inkling_rel_attn_decode(ctypes.byref(cache()), ctypes.byref(d), *a, FAKE, 1 << 30, None) == expect


def test_decode_pointers(lib):
    c, d = cache(), dec()
    n = lib.inkling_rel_attn_decode_workspace_size(ctypes.byref(c), ctypes.byref(d))
    assert n > 0
    # q, k_cache, v_cache, k_scale, v_scale, profiles, sink, block_table, lens, out, lse
    good = [FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]

    def call(change, c=c, d=d, ws=FAKE, size=n):
        a = list(good)
        for i, v in change.items():
            a[i] = v
        return lib.inkling_rel_attn_decode(ctypes.byref(c), ctypes.byref(d), *a, ws, size, None)

    for i in (0, 1, 2, 5, 7, 8, 9, 10):
        assert call({i: None}) == 1, i
    for i in (0, 1, 2, 5, 9):
        assert call({i: MIS}) == 1, i
    for i in (6, 7, 8, 10):
        assert call({i: ctypes.c_void_p(0x10002)}) == 1, i
    assert call({3: FAKE}) == 1 and call({3: FAKE, 4: FAKE}) == 1       # scales of a BF16 cache
    assert call({3: FAKE}, c=cache(dtype=1)) == 1                       # half the scales of an e4m3 one
    assert call({}, c=cache(dtype=1)) == 1
    assert call({}, d=dec(rel_extent=0)) == 1                           # profiles without an extent
    assert call({}, ws=None) == 1 and call({}, size=n - 1) == 1 and call({}, ws=MIS) == 1
    # no requests: nothing to do, nothing to launch
    assert lib.inkling_rel_attn_decode(ctypes.byref(c), ctypes.byref(dec(requests=0, rel_extent=0)), *([None] * 11),
                                       None, 0, None) == 0


def test_append_refusals(lib):
    from learned_relative_gqa_b200.binding import KVAppendDims

    # k, v, slots, k_scale, v_scale, clip_scale, tau, k_cache, v_cache
    def call(change=(), c=None, tokens=5, k_row=512, v_row=512, clip=0, thr=0.0):
        a = [FAKE, FAKE, FAKE, None, None, None, None, FAKE, ctypes.c_void_p(0x20000)]
        for i, v in dict(change).items():
            a[i] = v
        c = cache() if c is None else c
        return lib.inkling_kv_append(ctypes.byref(c), ctypes.byref(KVAppendDims(tokens, k_row, v_row, clip, thr)), *a,
                                     None)

    for i in (0, 1, 2, 7, 8):
        assert call({i: None}) == 1, i
    for i in (0, 1, 7, 8):
        assert call({i: MIS}) == 1, i
    assert call({2: ctypes.c_void_p(0x10004)}) == 1
    assert call({8: FAKE}) == 1                                          # one pool for both
    assert call(tokens=-1) == 1
    assert call(k_row=511) == 1 and call(v_row=516) == 1 and call(k_row=256) == 1
    assert call({5: FAKE}) == 1 and call({6: FAKE}) == 1                 # clip arguments without the clip
    assert call({5: MIS}, clip=1, thr=1.0) == 1
    assert call(clip=1, thr=-1.0) == 1 and call(clip=1, thr=float("nan")) == 1
    assert call({3: FAKE, 4: FAKE}) == 1 and call(c=cache(dtype=1)) == 1 and call({3: FAKE}, c=cache(dtype=1)) == 1
    assert call(tokens=1 << 31) == 2 and call(tokens=1 << 30) == 2 and call(k_row=1 << 59) == 2
    assert lib.inkling_kv_append(ctypes.byref(cache()), None, *([FAKE] * 9), None) == 1
    assert call({0: None, 1: None, 2: None}, tokens=0) == 0


def test_plan_refusals(lib):
    from learned_relative_gqa_b200.binding import KVPlanDims

    def at(i):
        return ctypes.c_void_p(0x1000000 * (i + 1))

    # old, new, table, free_pages, free_count, lens, query_start, slots, positions, info
    def call(change=(), **kw):
        d = dict(requests=4, page_size=16, max_pages=10, num_pages=50, max_tokens=100)
        d.update(kw)
        a = [at(i) for i in range(10)]
        for i, v in dict(change).items():
            a[i] = v
        return lib.inkling_kv_plan(ctypes.byref(KVPlanDims(**d)), *a, None)

    for i in range(10):
        assert call({i: None}) == 1, i
        assert call({i: ctypes.c_void_p(0x1000000 * (i + 1) + (4 if i == 7 else 2))}) == 1, i
    for kw, want in ((dict(requests=-1), 1), (dict(page_size=0), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1),
                     (dict(max_tokens=-1), 1), (dict(requests=16385), 2), (dict(max_pages=1 << 28), 2),
                     (dict(num_pages=1 << 31), 2), (dict(max_tokens=(1 << 30) + 1), 2),
                     (dict(requests=16384, max_pages=1 << 13), 2)):
        assert call(**kw) == want, kw
    # an output over an input: each pair is refused, also where only the ends meet
    for o in (5, 6, 7, 8, 9):
        for i in range(5):
            assert call({o: at(i)}) == 1, (o, i)
    assert call({5: ctypes.c_void_p(at(0).value + 12)}) == 1
    assert call({3: at(2)}) == 1                                         # table over the free pages


def test_python_wrappers_refuse_wrong_tensors(lib):
    """The checks that need no GPU: shapes, dtypes and devices of CPU tensors."""
    from learned_relative_gqa_b200 import binding
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.make_kv_cache_desc(k, k)
    with pytest.raises(ValueError, match="one shape"):
        binding.make_kv_cache_desc(k, k[:3])
    with pytest.raises(ValueError, match="bfloat16 or"):
        binding.make_kv_cache_desc(k.float(), k.float())
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.kv_plan(t[:, 0], t[:, 0], t, t[0], t[0, :1], page_size=16, num_pages=3, max_tokens=4)
    with pytest.raises(TypeError, match="old_lens must be a tensor"):
        binding.kv_plan([1, 2], t[:, 0], t, t[0], t[0, :1], page_size=16, num_pages=3, max_tokens=4)
    with pytest.raises(TypeError):
        binding.kv_plan(t[:, 0], t[:, 0], t, t[0], t[0, :1], page_size="16", num_pages=3, max_tokens=4)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.kv_append(k[0, :, :1], k[0, :, :1], torch.zeros(16, dtype=torch.int64), k, k)
    with pytest.raises(ValueError, match="one shape"):
        binding.kv_append(k[0], k[0], torch.zeros(16, dtype=torch.int64), k, k.float())
    with pytest.raises(ValueError, match="bfloat16 or"):
        binding.paged_decode(k[0], k.float(), k.float(), t, t[:, 0])
    with pytest.raises(ValueError, match="same strides"):
        binding.paged_decode(k[0], k.clone().transpose(0, 1).contiguous().transpose(0, 1), k, t, t[:, 0])
    with pytest.raises(TypeError, match="lens must be a tensor"):
        binding.paged_decode(k[0], k, k, t, None)
    from learned_relative_gqa_b200.paged import PagedKVCache
    with pytest.raises(ValueError, match="positive"):
        PagedKVCache(max_requests=1, max_len=0, num_pages=1, page_size=16, heads_kv=1, head_dim=64, device="cpu")
    with pytest.raises(ValueError, match="bfloat16 or"):
        PagedKVCache(max_requests=1, max_len=9, num_pages=1, page_size=16, heads_kv=1, head_dim=64,
                     dtype=torch.float16, device="cpu")
