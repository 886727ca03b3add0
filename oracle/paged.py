"""FP64 / integer oracle of the paged key-value cache operators: plain loops from the
definitions, sharing no code with the CUDA path. Test infrastructure only."""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 e4m3 codes (1 sign, 4 exponent, 3 mantissa bits, bias 7; 0x7f / 0xff: NaN)."""
    v = np.empty(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        v[c] = np.nan if e == 15 and m == 7 else sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return v


def plan(old, new, table, free, count, page, max_tokens, num_pages):
    """The page plan, one request after another. ``table`` and ``free`` (int arrays) are copied."""
    table, free = np.array(table), np.array(free)
    N, M = table.shape
    clamp = lambda x: min(max(int(x), 0), M * page)  # noqa: E731
    old, new = [clamp(x) for x in old], [clamp(x) for x in new]
    held = [-(-x // page) for x in old]
    want = [-(-x // page) for x in new]
    stack = [int(x) for x in free[:min(max(int(count), 0), num_pages)]]
    for r in range(N):
        for i in range(want[r], held[r]):
            if len(stack) < num_pages:
                stack.append(int(table[r, i]))
    short = taken = 0
    lens, slots, positions, start = [], [], [], [0]
    for r in range(N):
        have = held[r]
        for i in range(held[r], want[r]):
            if stack:
                table[r, i] = stack.pop()
                have += 1
                taken += 1
            else:
                short += 1
        lens.append(new[r] if new[r] <= old[r] else min(new[r], have * page))
        for pos in range(old[r], new[r]):
            p = int(table[r, pos // page]) if pos // page < have else -1
            slots.append(p * page + pos % page if 0 <= p < num_pages else -1)
            positions.append(pos)
        start.append(start[-1] + max(0, new[r] - old[r]))
    total = len(slots)
    slots, positions = slots[:max_tokens], positions[:max_tokens]
    slots += [-1] * (max_tokens - len(slots))
    positions += [0] * (max_tokens - len(positions))
    free[:len(stack)] = stack
    return dict(block_table=table, free_pages=free, lens=np.array(lens, dtype=np.int64), slots=np.array(slots, dtype=np.int64),
                positions=np.array(positions, dtype=np.int64), query_start=np.array(start),
                info=np.array([len(stack), total, short, taken]))


def decode(q, k, v, table, lens, profiles=None, sink=None, window=0, scale=None):
    """out [N,Hq,D], lse [N,Hq] and, for error bounds, [N,Hq,2]: the largest scale * sum |q||k| and |z| of each row.

    ``k``, ``v`` are FP64 pools [pages, page, Hkv, D] (decoded and scaled)."""
    N, Hq, D = q.shape
    pages, page, Hkv, _ = k.shape
    M = table.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    mag = np.zeros((N, Hq, 2))
    for n in range(N):
        L = min(max(int(lens[n]), 0), M * page)
        js = [j for j in range(max(0, L - window) if window else 0, L) if 0 <= table[n, j // page] < pages]
        at = [(int(table[n, j // page]), j % page) for j in js]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            sk = -np.inf if sink is None else float(sink[n, h])
            if not js:
                lse[n, h] = sk
                continue
            kk = np.array([k[p, o, g] for p, o in at])
            vv = np.array([v[p, o, g] for p, o in at])
            z = scale * (kk @ q[n, h])
            d = L - 1 - np.array(js)
            if profiles is not None:
                R = profiles.shape[2]
                z = z + np.where(d < R, profiles[n, h][np.minimum(d, R - 1)], 0.0)
            finite = np.isfinite(z)
            mag[n, h] = (scale * (np.abs(kk) @ np.abs(q[n, h]))).max(), np.abs(z[finite]).max(initial=0.0)
            top = max(z.max(), sk)
            if top == -np.inf:
                continue
            e = np.exp(z - top)
            total = e.sum() + np.exp(sk - top)
            lse[n, h] = top + np.log(total)
            out[n, h] = (e @ vv) / total
    return out, lse, mag
