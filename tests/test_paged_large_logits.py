"""Single-token attention where the logits are so large that FP32 holds them in steps of 2 to 16.

Every key of a request has the same profile entry b and the same value v, and the later half of the keys
have 8 ln 2 more in their product: as much as a logit may pass the running maximum by before that moves.
Whatever the steps make of the weights, they are finite, so out = v and lse is b to the resolution."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# in units of log2 the first is below 2^24 (steps of 1), then two of each binade up to 2^29, of either sign
BIAS = [-9e6, -1.3e7, -1.7e7, 2.4e7, -3e7, -5e7, 6e7, -8e7, -1e8, -1.2e8, 1.3e8, -1.5e8, -1.75e8, 1e8, -2.5e8, -3.5e8]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from learned_relative_gqa_b200 import build
    build.build()


@pytest.mark.parametrize("hq", [8, 16])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.bfloat16])
def test_decode_of_large_logits_stays_finite(dtype, split, hq):
    """v to 2^-16: the sums' (L / 8 + 64) 2^-24 twice, 1024 keys, and the terms of a probability, 2^-22."""
    from learned_relative_gqa_b200 import binding
    L, D, page = 1024, 64, 64
    N = 2  # hq heads of each: all of BIAS in either case
    M = 16 * (64 if split else 1)
    kc = torch.zeros(2 * 16, page, 1, D, device="cuda")
    table = torch.full((N, M), -1, dtype=torch.int32, device="cuda")
    table[:, :16] = torch.arange(32, device="cuda").view(2, 16)
    kc.view(2, L, D)[:, L // 2:, 0] = 1
    vc = torch.full_like(kc, 1.5)
    q = torch.zeros(N, hq, D, device="cuda")
    q[:, :, 0] = 1
    b = torch.tensor([BIAS[(n * hq + h) % 16] for n in range(N) for h in range(hq)], device="cuda").to(torch.bfloat16)
    prof = b.view(N, hq, 1).expand(N, hq, L).contiguous()
    one = torch.ones(1, device="cuda")
    scales = dict(k_scale=one, v_scale=one) if dtype == torch.float8_e4m3fn else {}
    out, lse = binding.paged_decode(q.to(torch.bfloat16), kc.to(dtype), vc.to(dtype), table,
                                    torch.tensor([L] * N, dtype=torch.int32, device="cuda"), prof,
                                    scale=8 * math.log(2.0), **scales)
    b = b.double().view(N, hq)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert (out - 1.5).abs().max() <= 1.5 * 2.0 ** -16
    # the sum's logarithm, and steps of the product b log2 e, of the sum and of the way back
    assert ((lse - b).abs() <= math.log(L) + 8 * math.log(2.0) + 16 * U * b.abs()).all()


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.bfloat16])
@pytest.mark.parametrize("split", [False, True])
def test_profile_rows_of_the_lowest_value_leave_no_key(dtype, split):
    """BF16's lowest value is beyond what logits in units of log 2 hold: a row of it is a row without keys."""
    from learned_relative_gqa_b200 import binding
    g = torch.Generator("cuda").manual_seed(1)
    N, hq, L, D, page = 2, 4, 300, 128, 16
    kc, vc = (torch.randn(2 * 19, page, 1, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    table = torch.full((N, 19 + (1000 if split else 0)), -1, dtype=torch.int32, device="cuda")
    table[:, :19] = torch.arange(38, device="cuda").view(2, 19)
    q = torch.randn(N, hq, D, generator=g, device="cuda").to(torch.bfloat16)
    prof = torch.zeros(N, hq, 304, dtype=torch.bfloat16, device="cuda")
    prof[0, 1], prof[1, 3] = torch.finfo(torch.bfloat16).min, -math.inf
    one = torch.ones(1, device="cuda")
    scales = dict(k_scale=one, v_scale=one) if dtype == torch.float8_e4m3fn else {}
    lens = torch.tensor([L, L - 7], dtype=torch.int32, device="cuda")
    for sink in (None, torch.randn(N, hq, generator=g, device="cuda"), torch.full((N, hq), torch.finfo(torch.float32).min, device="cuda")):
        out, lse = binding.paged_decode(q, kc, vc, table, lens, prof, sink, **scales)
        for n, h in ((0, 1), (1, 3)):
            assert not out[n, h].any()
            assert lse[n, h] == (-math.inf if sink is None else sink[n, h])
        assert torch.isfinite(out).all() and out[0, 0].any() and out[1, 1].any()
