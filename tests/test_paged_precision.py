"""Single-token attention: what its 16-bit terms of a probability p keep (three BF16 terms, two FP16 terms of
2^7 p for e4m3 caches), on problems where a lost term or a lost exponent range shows.

Keys and queries are zero, so logits are profile entries, exact in BF16, and keys with large p have v = 0,
so the result is the other keys' alone and its error is relative to that. Tolerances (u = 2^-24), relative:
* the terms: 2^-24 (BF16: three roundings of 2^-8), 2^-22 (FP16: two of 2^-11), and 2^-32 / p at most where
  the lifted FP16 terms end (2^-25 / 2^7 of the largest p);
* the exponential: 2^-22, and the product z log2 e before it: 2 u |z|;
* the products' sums: the tensor pipe cuts off, less than 2^-22 for each of at most four products into one sum;
* sums of a lane, between lanes and parts, the division: (L / 8 + 16) u, as all terms have one sign.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from learned_relative_gqa_b200 import build
    build.build()


def run(bias, small, dtype, hq, D, split):
    """bias [hq, L] by key; v is 3 for keys in ``small`` [L] and 0 for the others. Returns out / 3 [hq, D], lse."""
    from learned_relative_gqa_b200 import binding
    L, page = bias.shape[1], 16
    R = (L + 7) // 8 * 8
    prof = torch.zeros(1, hq, R, device="cuda")
    prof[0, :, :L] = bias.cuda().flip(1)  # by distance
    assert torch.equal(prof.to(torch.bfloat16).float(), prof)
    pages = -(-L // page)
    M = pages + (2048 if split else 0)
    table = torch.full((1, M), -1, dtype=torch.int32, device="cuda")
    table[0, :pages] = torch.arange(pages, device="cuda")
    kc = torch.zeros(pages, page, 1, D, device="cuda")
    vc = torch.zeros_like(kc)
    vc.view(-1, D)[:L][small.cuda()] = 3.0
    one = torch.ones(1, device="cuda")
    scales = dict(k_scale=one, v_scale=one) if dtype == torch.float8_e4m3fn else {}
    out, lse = binding.paged_decode(torch.zeros(1, hq, D, dtype=torch.bfloat16, device="cuda"), kc.to(dtype),
                                    vc.to(dtype), table, torch.tensor([L], dtype=torch.int32, device="cuda"),
                                    prof.to(torch.bfloat16), **scales)
    return out[0].cpu().double().numpy() / 3, lse[0].cpu().double().numpy()


def exact(bias, small):
    p = np.exp(bias.double().numpy())
    total = p.sum(1)
    return (p * small.numpy()).sum(1) / total, np.log(total)


def rounded(x, dtype):
    return torch.tensor(x).to(dtype).double().numpy()


FORMS = [(dtype, hq, D, split) for dtype in (torch.bfloat16, torch.float8_e4m3fn) for hq in (8, 16) for D in (64, 128)
         for split in (False, True)]


@pytest.mark.parametrize("dtype,hq,D,split", FORMS)
def test_every_term_of_a_probability_counts(dtype, hq, D, split):
    """Logits whose probability is worst for one term less: BF16, two terms are off by nearly 2^-17."""
    z = -np.arange(1, 400) / 256  # BF16 values down to -1.56
    z = rounded(z, torch.bfloat16)
    p = np.exp(z)
    if dtype == torch.bfloat16:
        first = rounded(p, dtype)
        lost = p - first - rounded(p - first, dtype)
    else:
        lost = p - rounded(p, torch.float16)
    lost = np.abs(lost) / p
    worst = np.argsort(-lost)[:hq]
    L = 17
    bias = torch.tensor(z[worst])[:, None].repeat(1, L).float()
    bias[:, 0] = 0
    small = torch.arange(L) > 0
    got, lse = run(bias, small, dtype, hq, D, split)
    want, l_want = exact(bias, small)
    tol = 2.0 ** -22 + 2.0 ** -22 + 2 * U * 1.6 + 4 * 2.0 ** -22 + (L / 8 + 16) * U
    assert lost[worst].min() > 2 * tol  # one term less would not pass
    assert (np.abs(got - want[:, None]) <= tol * want[:, None]).all(), np.abs(got / want[:, None] - 1).max() / tol
    assert (np.abs(lse - l_want) <= 2.0 ** -22 + (L / 8 + 16) * U + 4 * U * 3).all()


@pytest.mark.parametrize("L", [400, 1000])
@pytest.mark.parametrize("dtype,hq,D,split", FORMS)
def test_small_probabilities_beside_a_large_one_are_kept(dtype, hq, D, split, L):
    """A key of probability 1 in every 16, so in every tile, and e^-17.375 = 2^-25.07 for the others, which
    FP16 without the lift would round to nothing."""
    bias = torch.full((hq, L), -17.375)
    bias[:, ::16] = 0
    small = torch.arange(L) % 16 != 0
    got, lse = run(bias, small, dtype, hq, D, split)
    want, l_want = exact(bias, small)
    tol = 2.0 ** -22 + 2.0 ** -22 + 2 * U * 17.375 + 4 * 2.0 ** -22 + (L / 8 + 16) * U
    if dtype == torch.float8_e4m3fn:
        assert not rounded(math.exp(-17.375), torch.float16).any()
        tol += 2.0 ** -32 / math.exp(-17.375)
    assert tol < 0.01  # the keys' loss, or that of half of them, would not pass
    assert (np.abs(got - want[:, None]) <= tol * want[:, None]).all(), np.abs(got / want[:, None] - 1).max() / tol
    assert (np.abs(lse - l_want) <= 2.0 ** -22 + (L / 8 + 64) * U + 4 * U * np.abs(l_want)).all()
