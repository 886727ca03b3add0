"""GPU paged-cache operators against their FP64 / integer oracle, at the sizes and masks
where they can go wrong.

Tolerances of the attention, per row, from the arithmetic (u = 2^-24, half an FP32 step):
* a logit: D products summed in FP32, dz = (D + 16) u sum|q||k| scale + 4 u |z|
  (``mag`` of the oracle holds both; the factor 4 covers the products with the scale and
  log2 e and the bias, one rounding each);
* a probability: 2 dz relative (value and maximum), the exponential's 2^-22, and in the
  second product its two-part form, off by at most 2^-8 of 2^-8 of it (BF16; FP16 is finer);
* sums over the keys: a lane adds a sixteenth of a part's keys one after the other, and
  then at most 64 more partial sums are added, (L / 8 + 64) u with room for both sums.
out: max|v| (2^-16 + 2 (2 dz + 2^-22) + 2 (L / 8 + 64) u), as numerator and denominator
both carry the last two terms. lse: dz + 2^-22 + (L / 8 + 64) u + 4 u |lse|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import l2clip as clip_ref
from oracle import paged as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from learned_relative_gqa_b200 import build
    build.build()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def make_cache(num_pages, page, hkv, d, dtype, layout, g):
    shape = (num_pages, hkv, page, d) if layout == "hnd" else (num_pages, page, hkv, d)
    x = torch.randn(shape, generator=g, device="cuda")
    scale = None
    if dtype == "e4m3":
        scale = 0.01 + 0.02 * torch.rand(hkv, generator=g, device="cuda")
        x = (x / (scale[:, None, None] if layout == "hnd" else scale[:, None])).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        x = x.to(torch.bfloat16)
    return (x.transpose(1, 2) if layout == "hnd" else x), scale


def bits(cache):
    return cache.view(torch.uint8 if cache.dtype == torch.float8_e4m3fn else torch.int16)


def problem(lens, hq, hkv, d, page, r, dtype="bf16", layout="nhd", seed=0, max_pages=None, poison=True, sink=True):
    """Random tensors of a decode call; every cached value that no request owns is NaN."""
    g = gen(seed)
    N = len(lens)
    need = [-(-x // page) for x in lens]
    M = max_pages or max(max(need), 1)
    total = sum(need)
    num_pages = total + 3
    kc, ks = make_cache(num_pages, page, hkv, d, dtype, layout, g)
    vc, vs = make_cache(num_pages, page, hkv, d, dtype, layout, g)
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((N, M), -1, dtype=torch.int32)
    at = 0
    owned = torch.zeros(num_pages, page, dtype=torch.bool)
    for n in range(N):
        table[n, :need[n]] = order[at:at + need[n]]
        for i in range(need[n]):
            owned[order[at + i].long(), :min(page, lens[n] - i * page)] = True
        at += need[n]
    if poison:
        for c in (kc, vc):
            nan = torch.tensor(float("nan"), device="cuda").to(c.dtype)
            b = bits(c)
            b[~owned.cuda()] = bits(nan.view(1))[0]
    x = dict(q=torch.randn(N, hq, d, generator=g, device="cuda").to(torch.bfloat16), k_cache=kc, v_cache=vc,
             block_table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             profiles=(0.5 * torch.randn(N, hq, r, generator=g, device="cuda")).to(torch.bfloat16) if r else None,
             sink=torch.randn(N, hq, generator=g, device="cuda") if sink else None)
    return x, dict(k_scale=ks, v_scale=vs)


def workspace(x, fill):
    from learned_relative_gqa_b200 import binding
    N, Hq, _ = x["q"].shape
    R = 0 if x["profiles"] is None else x["profiles"].shape[2]
    ws = binding.alloc_decode_workspace(binding.make_kv_cache_desc(x["k_cache"], x["v_cache"]),
                                        binding.DecodeDims(N, Hq, R, 0, x["block_table"].shape[1], 0.0), "cuda")
    return ws.fill_(fill)


def f64(t):
    return None if t is None else t.cpu().double().numpy()


def pool64(cache, scale):
    x = f64(cache)
    return x if scale is None else x * f64(scale)[:, None]


def check(x, scales, window=0, scale=None, got=None):
    from learned_relative_gqa_b200 import binding
    out, lse = got or binding.paged_decode(**x, **scales, window=window, scale=scale)
    torch.cuda.synchronize()
    k, v = pool64(x["k_cache"], scales["k_scale"]), pool64(x["v_cache"], scales["v_scale"])
    o_ref, l_ref, mag = ref.decode(f64(x["q"]), k, v, x["block_table"].cpu().numpy(), x["lens"].cpu().numpy(),
                                   f64(x["profiles"]), f64(x["sink"]), window, scale)
    D, L = x["q"].shape[2], max(1, int(x["lens"].max()))
    dz = (D + 16) * U * mag[:, :, 0] + 4 * U * mag[:, :, 1]
    vmax = np.nanmax(np.abs(v)) if np.isfinite(v).any() else 0.0
    o_tol = vmax * (2.0 ** -16 + 2 * (2 * dz + 2.0 ** -22) + 2 * (L / 8 + 64) * U)
    finite = np.isfinite(l_ref)
    l_tol = dz + 2.0 ** -22 + (L / 8 + 64) * U + 4 * U * np.abs(np.where(finite, l_ref, 0.0))
    out, lse = f64(out), f64(lse)
    assert np.isfinite(out).all()
    assert (np.abs(out - o_ref) <= o_tol[:, :, None]).all(), float((np.abs(out - o_ref) - o_tol[:, :, None]).max())
    assert np.array_equal(finite, np.isfinite(lse)) and np.array_equal(l_ref[~finite], lse[~finite])
    assert (np.abs(lse[finite] - l_ref[finite]) <= l_tol[finite]).all()
    return out, lse


DECODE = [  # lens, hq, hkv, d, page, r, window, dtype, layout
    ([1], 1, 1, 64, 1, 0, 0, "bf16", "nhd"),
    ([128], 4, 2, 64, 16, 64, 0, "bf16", "nhd"),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65, 0], 8, 2, 128, 16, 8, 0, "bf16", "nhd"),
    ([0, 1, 31, 32, 33, 127, 128, 129, 300], 8, 1, 128, 16, 16, 0, "e4m3", "nhd"),
    ([700, 3, 257], 6, 2, 128, 24, 64, 0, "bf16", "hnd"),          # a page size that no tile divides
    ([700, 3, 257], 6, 2, 64, 7, 4096, 0, "e4m3", "hnd"),          # profile longer than every request
    ([513, 40], 12, 1, 128, 64, 128, 0, "bf16", "nhd"),            # 12 heads to a KV head: two groups of 8
    ([513, 40], 16, 1, 64, 64, 128, 0, "bf16", "hnd"),
    ([300, 140], 20, 1, 128, 32, 40, 0, "bf16", "nhd"),            # 20: two blocks of heads
    ([300, 140], 33, 1, 64, 32, 40, 0, "e4m3", "nhd"),             # 33: three, the last with one head
    ([900, 1, 511, 512, 513], 16, 4, 128, 16, 512, 512, "bf16", "nhd"),
    ([900, 1, 511, 100, 513], 4, 4, 64, 16, 64, 1, "bf16", "hnd"),  # a window of the token itself
    ([900, 90, 5], 8, 2, 128, 128, 256, 100, "e4m3", "hnd"),       # a window that begins inside a page
    ([2500], 8, 8, 128, 16, 128, 0, "bf16", "nhd"),                # one request over many CTAs
    ([3001], 8, 1, 128, 64, 1000, 0, "e4m3", "nhd"),
    ([17] * 150 + [0] * 20 + [400], 2, 1, 64, 16, 8, 0, "bf16", "nhd"),  # more requests than threads of a block
]


@pytest.mark.parametrize("lens,hq,hkv,d,page,r,window,dtype,layout", DECODE)
def test_decode(lens, hq, hkv, d, page, r, window, dtype, layout):
    x, s = problem(lens, hq, hkv, d, page, r, dtype, layout, seed=len(lens) + hq + d)
    out, lse = check(x, s, window)
    for n, L in enumerate(lens):
        if L == 0:
            assert not out[n].any() and np.array_equal(lse[n], f64(x["sink"])[n])


def random_case(seed):
    rng = np.random.default_rng(seed)
    hkv = int(rng.choice([1, 2, 3, 5]))
    group = int(rng.choice([1, 2, 3, 4, 7, 8, 9, 16, 17]))
    n = int(rng.choice([1, 2, 5, 17, 40]))
    most = int(rng.choice([40, 300, 1500 if n < 10 else 300]))
    lens = [int(x) if rng.random() < 0.9 else 0 for x in rng.integers(1, most + 1, n)]
    page = int(rng.choice([1, 3, 8, 16, 17, 24, 32, 40, 64, 500, 2048]))
    return dict(lens=lens, hq=hkv * group, hkv=hkv, d=int(rng.choice([64, 128])), page=page,
                r=8 * int(rng.choice([0, 1, 5, 40, 300])), dtype=str(rng.choice(["bf16", "e4m3"])),
                layout=str(rng.choice(["nhd", "hnd"])), seed=seed,
                max_pages=max(1, -(-max(lens + [1]) // page)) + int(rng.choice([0, 3, 2000 // page + 1])),
                sink=bool(rng.random() < 0.8)), int(rng.choice([0, 0, 1, 7, 64, 200]))


@pytest.mark.parametrize("seed", range(40))
def test_decode_random_shapes(seed):
    kw, window = random_case(seed)
    x, s = problem(**kw)
    check(x, s, window)


@pytest.mark.parametrize("hq,hkv,d,dtype", [(16, 1, 128, "bf16"), (16, 1, 64, "e4m3"), (4, 2, 128, "e4m3"),
                                            (40, 2, 64, "bf16")])
@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 1], [5, 0, 40, 1, 1, 0, 2], [33] * 40])
def test_decode_short_requests_under_a_long_table(hq, hkv, d, dtype, lens):
    """The table allows 8192 tokens, so the split form runs, with next to nothing to split."""
    x, s = problem(lens, hq, hkv, d, 16, 8, dtype, seed=21, max_pages=512)
    check(x, s)


@pytest.mark.parametrize("hq,hkv,d,dtype", [(2, 1, 64, "bf16"), (16, 1, 128, "bf16"), (8, 1, 128, "e4m3"),
                                            (9, 1, 64, "e4m3")])
def test_decode_one_request_over_all_workers(hq, hkv, d, dtype):
    """Long chains of parts, joined by whole blocks."""
    x, s = problem([20011], hq, hkv, d, 64, 256, dtype, seed=22)
    check(x, s)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_many_units_without_a_split(dtype):
    """A table of few tiles and more units than CTAs on the device: both sides of the limit of the whole form."""
    for n in (256, 257):
        x, s = problem([(7 * i) % 50 for i in range(n)], 4, 2, 64, 16, 8, dtype, seed=n)
        check(x, s)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_scale_and_no_sink(dtype):
    x, s = problem([100, 0, 7], 4, 2, 128, 16, 0, dtype, seed=5, sink=False)
    _, lse = check(x, s, scale=0.3)
    assert np.isneginf(lse[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_entries_outside_the_pool_are_masked(dtype):
    x, s = problem([200, 64, 16], 4, 2, 128, 16, 32, dtype, seed=6)
    t = x["block_table"]
    num_pages = x["k_cache"].shape[0]
    t[0, 3], t[0, 7], t[0, 12], t[1, 0] = -1, num_pages, 2 ** 31 - 1, -2 ** 31
    t[2, 0] = num_pages  # this request keeps no key
    out, lse = check(x, s)
    assert not out[2].any() and np.array_equal(lse[2], f64(x["sink"])[2])


def test_decode_does_not_read_entries_outside_the_window_or_the_length():
    """Their pages hold NaN; a bad page number there changes nothing either."""
    x, s = problem([500, 77], 4, 2, 128, 16, 64, seed=7, max_pages=40)
    a = check(x, s, window=60)
    t = x["block_table"]
    t[0, :27] = 0
    t[0, 32:] = 10 ** 9
    t[1, 5:] = -5
    b = check(x, s, window=60)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_decode_lengths_outside_the_table():
    x, s = problem([64, 64, 64], 4, 2, 64, 16, 8, seed=8)
    x["lens"] = torch.tensor([2 ** 31 - 1, -7, 64], dtype=torch.int32, device="cuda")
    from learned_relative_gqa_b200 import binding
    out, lse = binding.paged_decode(**x, **s)
    x["lens"] = torch.tensor([64, 0, 64], dtype=torch.int32, device="cuda")
    check(x, s, got=(out, lse))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_profiles_that_mask(dtype):
    """-inf and the type's lowest value in the profile take keys out, without NaN; a row may lose all."""
    x, s = problem([300, 40], 4, 2, 128, 16, 64, dtype, seed=9)
    low = torch.finfo(torch.bfloat16).min
    x["profiles"][0, 0, 3:50] = -math.inf
    x["profiles"][0, 1, :] = low
    x["profiles"][1, 2, :] = -math.inf  # 40 tokens, 64 entries: nothing is left but the sink
    out, lse = check(x, s)
    assert not out[1, 2].any() and abs(lse[1, 2] - float(x["sink"][1, 2])) < 1e-6
    x["sink"] = None
    out, lse = check(x, s)
    assert not out[1, 2].any() and np.isneginf(lse[1, 2])


def test_decode_propagates_nan_of_an_allowed_key_to_its_group_only():
    x, s = problem([200, 100], 8, 2, 128, 16, 16, seed=10)
    p = int(x["block_table"][0, 4])
    x["k_cache"][p, 5, 1, 3] = float("nan")
    from learned_relative_gqa_b200 import binding
    out, lse = binding.paged_decode(**x, **s)
    assert torch.isnan(out[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_large_logits_move_the_maximum(dtype):
    """Later keys far above earlier ones (the running maximum moves, O is rescaled) and far below."""
    for sign in (1.0, -1.0):
        x, s = problem([400], 8, 2, 64, 16, 400, dtype, seed=11)
        ramp = sign * torch.linspace(60, -60, 400, device="cuda")  # by distance: the newest first
        x["profiles"][:] = ramp.to(torch.bfloat16)
        check(x, s)


def test_decode_small_and_large_queries_e4m3():
    """q is brought to FP16 by a power of two per head: its scale must not matter."""
    x, s = problem([150], 4, 1, 128, 16, 0, "e4m3", seed=12)
    for h, f in enumerate((2.0 ** -60, 2.0 ** 12, 0.0, 1.0)):
        x["q"][0, h] *= f
    check(x, s, scale=2.0 ** -12)


def test_decode_scales_that_underflow_leave_masked_keys_masked():
    """A query of zeros with a tiny key scale, and a tiny logit scale: every logit is 0, and the keys
    behind the length still do not count."""
    x, s = problem([5, 33], 4, 1, 128, 16, 0, "e4m3", seed=23)
    x["q"].zero_()
    s["k_scale"].fill_(1e-30)
    check(x, s)
    y, t = problem([5, 33], 4, 1, 64, 16, 8, seed=24)
    check(y, t, scale=1e-300)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_decode_keeps_a_long_tail_of_small_probabilities(dtype):
    """One key with probability 1 and 5999 with e^-17.375 = 2^-25.07 of it each, all with the largest
    value: together they are 1.7e-4 of the result."""
    for lens in ([6000], [400], [6000, 5, 900]):
        x, s = problem(lens, 8, 1, 128, 64, 6000, dtype, seed=25, poison=False)
        x["q"].zero_()
        x["profiles"].fill_(-17.375)
        x["profiles"][:, :, 0] = 0
        x["sink"].fill_(-30.0)
        x["v_cache"].copy_(torch.full(x["v_cache"].shape, 448.0 if dtype == "e4m3" else 3.0, device="cuda"))
        check(x, s)


def test_decode_equal_calls_give_equal_bits():
    from learned_relative_gqa_b200 import binding
    x, s = problem([1500, 3, 700, 0], 16, 2, 128, 16, 64, seed=13)
    a = binding.paged_decode(**x, **s)
    ws = workspace(x, 0xAB)  # what a workspace holds means nothing
    for _ in range(5):
        b = binding.paged_decode(**x, **s, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_pool_beyond_32_bit_offsets():
    """Pages whose byte and element offsets pass 2^32."""
    from learned_relative_gqa_b200 import binding
    g = gen(14)
    hkv, d, page = 8, 128, 16
    num_pages = (1 << 32) // (hkv * d * page) + 64
    kc = torch.empty(num_pages, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    table = torch.tensor([[num_pages - 1, 3, num_pages - 9, num_pages // 2 + 1]], dtype=torch.int32, device="cuda")
    small = torch.randn(2, 4, page, hkv, d, generator=g, device="cuda").to(torch.bfloat16)
    slots = (table[0].long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
    binding.kv_append(small[0].reshape(-1, hkv, d), small[1].reshape(-1, hkv, d), slots, kc, vc)
    assert torch.equal(kc[table[0].long()], small[0]) and torch.equal(vc[table[0].long()], small[1])
    x = dict(q=torch.randn(1, 16, d, generator=g, device="cuda").to(torch.bfloat16), block_table=table,
             lens=torch.tensor([61], dtype=torch.int32, device="cuda"),
             profiles=torch.randn(1, 16, 8, generator=g, device="cuda").to(torch.bfloat16),
             sink=torch.randn(1, 16, generator=g, device="cuda"))
    got = binding.paged_decode(k_cache=kc, v_cache=vc, **x)
    x["block_table"] = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    check(dict(x, k_cache=small[0], v_cache=small[1]), dict(k_scale=None, v_scale=None), got=got)


def test_decode_on_another_stream_and_from_views():
    """A stream of its own, and pools that are slices of a wider allocation."""
    from learned_relative_gqa_b200 import binding
    x, s = problem([300, 20], 4, 2, 64, 16, 8, seed=15)
    both = torch.stack((x["k_cache"], x["v_cache"]), 1)  # [pages, 2, page, heads, d]
    x["k_cache"], x["v_cache"] = both[:, 0], both[:, 1]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = binding.paged_decode(**x, **s, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    check(x, s, got=got)


def test_decode_captured_and_replayed_with_other_lengths():
    from learned_relative_gqa_b200 import binding
    lens = [700, 5, 0, 257]
    x, s = problem(lens, 8, 2, 128, 16, 64, seed=16, poison=False)
    binding.paged_decode(**x, **s)
    graphs = []
    ws = workspace(x, 0)
    for window in (0, 100):  # two graphs that share a workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = binding.paged_decode(**x, **s, window=window, workspace=ws)
        graphs.append((g, window, got))
    for new in ([700, 5, 0, 257], [1, 0, 0, 3], [640, 4, 0, 250]):
        x["lens"].copy_(torch.tensor(new, dtype=torch.int32))
        for g, window, got in graphs + graphs:
            g.replay()
            check(x, s, window, got=got)


def test_decode_captured_with_forks_and_joins():
    """Two streams inside one capture, each with two calls, joined before a last one: launches that may
    overlap their predecessor must still wait for all that the capture orders before them."""
    from learned_relative_gqa_b200 import binding
    x, s = problem([900, 30, 0, 411], 8, 2, 64, 16, 32, seed=17)
    y, t = problem([350, 1200], 4, 1, 128, 32, 0, "e4m3", seed=18)
    for a, b in ((x, s), (y, t)):
        binding.paged_decode(**a, **b)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    got = {}
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got["a"] = binding.paged_decode(**x, **s)
        with torch.cuda.stream(side):
            got["b"] = binding.paged_decode(**y, **t)
            got["c"] = binding.paged_decode(**y, **t, window=100)
        got["d"] = binding.paged_decode(**x, **s, window=50)
        main.wait_stream(side)
        got["e"] = binding.paged_decode(**x, **s, window=7)
    for _ in range(3):
        for pair in got.values():
            for z in pair:
                z.fill_(float("nan"))
        g.replay()
        check(x, s, got=got["a"])
        check(y, t, got=got["b"])
        check(y, t, 100, got=got["c"])
        check(x, s, 50, got=got["d"])
        check(x, s, 7, got=got["e"])


def test_decode_waits_for_the_kernel_before_it():
    """Calls back to back with the kernels that write their inputs, and with kernels of other
    libraries between: each reads what was written last."""
    from learned_relative_gqa_b200 import binding
    x, s = problem([1500, 700, 20], 8, 2, 128, 16, 64, seed=19)
    want = binding.paged_decode(**x, **s)
    lens, q = x["lens"].clone(), x["q"].clone()
    wrong = torch.randn_like(x["q"].float()).to(torch.bfloat16)
    for _ in range(30):
        x["lens"].fill_(3)
        x["q"].copy_(wrong)
        binding.paged_decode(**x, **s)
        x["lens"].copy_(lens)
        x["q"].copy_(q)
        got = binding.paged_decode(**x, **s)
        again = binding.paged_decode(**x, **s)
        for a, b in ((got, want), (again, want)):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------
def e4m3_codes(x64):
    """Nearest code of each value (ties to the even one), saturated; NaN to NaN."""
    table = ref.e4m3_values()
    pos = table[:0x7f]
    a = np.minimum(np.abs(x64), 448.0)
    hi = np.searchsorted(pos, a).clip(0, 0x7e)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(x64), 0x80, 0)
    return np.where(np.isnan(x64), 0x7f, code).astype(np.uint8)


APPEND = [(1, 1, 64, 16, "bf16", "nhd"), (7, 3, 128, 5, "bf16", "hnd"), (257, 8, 128, 64, "bf16", "nhd"),
          (1, 1, 128, 1, "e4m3", "nhd"), (130, 5, 64, 16, "e4m3", "hnd"), (33, 2, 128, 24, "e4m3", "nhd")]


@pytest.mark.parametrize("T,H,D,page,dtype,layout", APPEND)
def test_append_copies_or_rounds_exactly(T, H, D, page, dtype, layout):
    from learned_relative_gqa_b200 import binding
    g = gen(T + H)
    num_pages = T // page + 3
    kc, ks = make_cache(num_pages, page, H, D, dtype, layout, g)
    vc, vs = make_cache(num_pages, page, H, D, dtype, layout, g)
    if ks is not None:  # powers of two, so that ties of the rounding occur; and large values saturate
        ks, vs = torch.full_like(ks, 0.125), torch.full_like(vs, 2.0 ** -8)
    kv = torch.randn(T, 2, H, D, generator=g, device="cuda").to(torch.bfloat16)
    kv[0, :, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0])
    k, v = kv[:, 0], kv[:, 1]  # rows of a fused projection
    slots = torch.randperm(num_pages * page, generator=g, device="cuda")[:T]
    if T > 5:
        slots[3], slots[5] = -1, num_pages * page  # outside the pool: skipped
    kb, vb = kc.clone(), vc.clone()
    binding.kv_append(k, v, slots, kc, vc, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    for x, before, after, s in ((k, kb, kc, ks), (v, vb, vc, vs)):
        want = bits(before).cpu().numpy().copy()
        if s is None:
            rows = x.contiguous().view(torch.int16).cpu().numpy()
        else:
            # the quotient is rounded to FP32 first; a power of two makes that exact
            rows = e4m3_codes(f64(x) / f64(s)[:, None])
        for t, slot in enumerate(slots.tolist()):
            if 0 <= slot < num_pages * page:
                want[slot // page, slot % page] = rows[t]
        got = bits(after).cpu().numpy()
        if s is not None:  # a NaN may carry either sign
            got, want = np.where(got == 0xff, 0x7f, got), np.where(want == 0xff, 0x7f, want)
        assert np.array_equal(got, want)


@pytest.mark.parametrize("scale", [0.0107, 1 / 3, 3.0, 1e-3, 7.7e-20, 5e21, 1.9e-37])
def test_append_e4m3_quotients_are_correctly_rounded(scale):
    """Every BF16 value, with scales that are no powers of two: the code is that of x / scale rounded
    to FP32 and then to e4m3."""
    from learned_relative_gqa_b200 import binding
    x = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16).view(-1, 1, 64)
    T = x.shape[0]
    kc = torch.zeros(T // 16, 16, 1, 64, dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.zeros_like(kc)
    s = torch.tensor([scale], device="cuda")
    binding.kv_append(x, x, torch.arange(T, device="cuda"), kc, vc, k_scale=s, v_scale=s)
    with np.errstate(all="ignore"):
        q = (x.cpu().float().numpy() / np.float32(scale)).astype(np.float64)
    want = e4m3_codes(q).reshape(-1)
    for c in (kc, vc):
        got = c.view(torch.uint8).cpu().numpy().reshape(-1)
        assert np.array_equal(np.where(got == 0xff, 0x7f, got), np.where(want == 0xff, 0x7f, want))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("with_scale,with_tau,thr", [(True, True, 8.0), (False, True, 5.0), (True, False, 1e9),
                                                     (False, False, 0.0)])
def test_append_clips_k_like_the_clip_of_its_own(D, with_scale, with_tau, thr):
    """Within half a BF16 step of the oracle's value plus 1e-5 of it (the FP32 arithmetic of the
    clip, as in the parity tests of the clip itself)."""
    from learned_relative_gqa_b200 import binding
    g = gen(D + with_scale)
    T, H, page = 53, 3, 16
    k = (3 * torch.randn(T, H, D, generator=g, device="cuda") * torch.rand(T, H, 1, generator=g, device="cuda")).to(torch.bfloat16)
    k[4] = 0
    v = torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16)
    scale = 0.5 + torch.rand(H, D, generator=g, device="cuda") if with_scale else None
    tau = 0.5 + 1.5 * torch.rand(T, generator=g, device="cuda") if with_tau else None
    kc = torch.zeros(5, page, H, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.randperm(5 * page, generator=g, device="cuda")[:T]
    binding.kv_append(k, v, slots, kc, vc, threshold=thr, clip_scale=scale, tau=tau)
    got = f64(kc.view(-1, H, D)[slots])
    want = clip_ref.forward(f64(k)[None], f64(scale), None if tau is None else f64(tau)[None], thr)[0]
    half = 0.5 * 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - 7)
    assert (np.abs(got - want) - half).max() <= 1e-5 * max(1.0, np.abs(want).max())
    assert torch.equal(vc.view(-1, H, D)[slots], v)


def test_append_of_no_rows_and_of_none_that_fit():
    from learned_relative_gqa_b200 import binding
    kc = torch.randn(2, 4, 1, 64, device="cuda").to(torch.bfloat16)
    vc, before = kc.clone(), kc.clone()
    k = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    binding.kv_append(k[:0], k[:0], torch.empty(0, dtype=torch.int64, device="cuda"), kc, vc)
    binding.kv_append(k, k, torch.tensor([-1, 8, 2 ** 62], device="cuda"), kc, vc)
    assert torch.equal(kc, before) and torch.equal(vc, before)


# --------------------------------------------------------------------------
# plan
# --------------------------------------------------------------------------
def run_plan(old, new, table, free, count, page, max_tokens, num_pages):
    from learned_relative_gqa_b200 import binding
    i32 = dict(dtype=torch.int32, device="cuda")
    t, f = torch.as_tensor(np.asarray(table)).to(**i32).contiguous(), torch.as_tensor(np.asarray(free)).to(**i32)
    p = binding.kv_plan(torch.tensor(old, **i32), torch.tensor(new, **i32), t, f, torch.tensor([count], **i32),
                        page_size=page, num_pages=num_pages, max_tokens=max_tokens)
    want = ref.plan(old, new, table, free, count, page, max_tokens, num_pages)
    got = dict(p, block_table=t, free_pages=f)
    for name in want:
        assert np.array_equal(got[name].cpu().numpy(), want[name]), name
    return want


def random_plan(N, page, M, seed, slack, max_new):
    rng = np.random.default_rng(seed)
    cap = M * page
    old = rng.integers(0, cap + 1, N) * (rng.random(N) < 0.8)
    new = np.minimum(cap, old + rng.integers(0, max_new + 1, N))
    cut = rng.random(N) < 0.3
    new = np.where(cut, rng.integers(0, cap + 1, N) % (old + 1), new)
    held, want = -(-old // page), -(-new // page)
    need = int(np.maximum(want - held, 0).sum())
    num_pages = int(held.sum()) + max(1, int(need * slack))
    order = rng.permutation(num_pages)
    table, at = np.full((N, M), -1), 0
    for r in range(N):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    free = np.full(num_pages, -1)
    free[:num_pages - at] = order[at:]
    return old.tolist(), new.tolist(), table, free, num_pages - at, page, num_pages


@pytest.mark.parametrize("N,page,M,max_new", [(1, 16, 8, 20), (3, 1, 40, 9), (64, 16, 32, 1), (200, 24, 16, 300),
                                              (513, 64, 4, 64), (1500, 16, 8, 40)])
@pytest.mark.parametrize("slack", [1.0, 0.4, 0.0])
def test_plan_random_lengths(N, page, M, max_new, slack):
    """With pages enough, with too few, and with none but those given back; more and fewer token
    entries than tokens."""
    for seed in range(2):
        old, new, table, free, count, page, num_pages = random_plan(N, page, M, 17 * N + seed, slack, max_new)
        total = sum(max(0, b - a) for a, b in zip(old, new))
        run_plan(old, new, table, free, count, page, total + 37 if seed else max(0, total - 5), num_pages)


def test_plan_edges():
    t = np.full((2, 3), -1)
    run_plan([0, 0], [0, 0], t, [0, 1, 2], 3, 4, 5, 3)             # nothing to do
    run_plan([0, 0], [12, 1], t, [0, 1, 2, 3], 4, 4, 13, 4)        # the last page
    run_plan([-5, 3], [10 ** 9, -1], [[-1] * 3, [2, -1, -1]], [0, 1, 7], 9, 4, 20, 3)  # lengths and count out of range
    run_plan([4], [5], [[1, -1, -1]], [5, 9], 2, 4, 1, 2)          # a free list that names no page of the pool
    run_plan([2], [3], [[77]], [0], 1, 4, 1, 1)                    # nor does the table
    run_plan([0], [3], [[-1]], [0], -3, 4, 0, 1)                   # no pages, no entries
    run_plan([], [], np.zeros((0, 3), dtype=int), [0, 1], 2, 4, 3, 2)  # no requests


def test_plan_largest_batch():
    old, new, table, free, count, page, num_pages = random_plan(16384, 16, 4, 5, 0.8, 30)
    run_plan(old, new, table, free, count, page, 300000, num_pages)
