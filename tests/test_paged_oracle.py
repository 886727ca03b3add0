"""Pins of the paged-cache oracle (oracle/paged.py): cases worked by hand, and the
attention oracle of the whole sequence."""
import numpy as np
import torch

import oracle
from oracle import paged as ref


def test_e4m3_table_is_the_format():
    v = ref.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    assert v[0x7e] == 448.0 and v[1] == 2.0 ** -9 and v[0x38] == 1.0


def test_plan_worked_by_hand():
    # pages of 4; row 0 grows 3 -> 6, row 1 ends, row 2 starts with 5, row 3 is cut from 9 to 4
    table = np.array([[10, -1, -1], [20, 21, -1], [-1, -1, -1], [30, 31, 32]])
    free = np.full(50, -1)
    free[:2] = [40, 41]
    p = ref.plan([3, 5, 0, 9], [6, 0, 5, 4], table, free, 2, 4, 10, 50)
    # returned: 20 21 31 32 on top of 40 41; taken from the top: 32 (row 0), 31 21 (row 2)
    assert p["block_table"].tolist() == [[10, 32, -1], [20, 21, -1], [31, 21, -1], [30, 31, 32]]
    assert p["free_pages"][:3].tolist() == [40, 41, 20] and p["info"].tolist() == [3, 8, 0, 3]
    assert p["lens"].tolist() == [6, 0, 5, 4] and p["query_start"].tolist() == [0, 3, 3, 8, 8]
    assert p["slots"].tolist() == [43, 128, 129, 124, 125, 126, 127, 84, -1, -1]
    assert p["positions"].tolist() == [3, 4, 5, 0, 1, 2, 3, 4, 0, 0]


def test_plan_without_enough_pages():
    p = ref.plan([2, 0], [9, 4], np.array([[7, -1, -1], [-1, -1, -1]]), np.array([3] + [-1] * 9), 1, 4, 11, 10)
    assert p["lens"].tolist() == [8, 0] and p["info"].tolist() == [0, 11, 2, 1]
    assert p["slots"].tolist() == [30, 31, 12, 13, 14, 15, -1, -1, -1, -1, -1]


def test_decode_is_the_last_row_of_the_whole_sequence():
    rng = np.random.default_rng(3)
    for L, W, R in ((37, 0, 16), (37, 11, 16), (5, 0, 64), (1, 0, 8), (40, 9, 0)):
        Hq, Hkv, D, P = 4, 2, 64, 8
        q, k, v = rng.normal(size=(1, L, Hq, D)), rng.normal(size=(1, L, Hkv, D)), rng.normal(size=(1, L, Hkv, D))
        prof, sink = rng.normal(size=(1, Hq, L, R)), rng.normal(size=(1, L, Hq))
        ones = np.ones((1, L), dtype=np.uint8)
        o, l, _ = oracle.forward(q, k, v, prof, sink, ones, window=W)
        pages = rng.permutation(12)[:-(-L // P)]
        kc, vc = np.full((12, P, Hkv, D), np.nan), np.full((12, P, Hkv, D), np.nan)
        for j in range(L):
            kc[pages[j // P], j % P], vc[pages[j // P], j % P] = k[0, j], v[0, j]
        got, lse, _ = ref.decode(q[:, -1], kc, vc, pages[None], [L], prof[:, :, -1] if R else None, sink[:, -1], W)
        assert np.abs(got[0] - o[0, -1]).max() < 1e-12 and np.abs(lse[0] - l[0, -1]).max() < 1e-12


def test_decode_without_allowed_keys():
    k = np.ones((2, 4, 1, 64))
    out, lse, _ = ref.decode(np.ones((3, 2, 64)), k, k, np.array([[0], [5], [-1]]), [0, 3, 2], None,
                             np.array([[1.0, 2.0]] * 3))
    assert not out.any() and np.array_equal(lse, [[1.0, 2.0]] * 3)
