"""Cases of the paged key-value cache operators: the page plan of a serving step, the
append of new key and value rows to the cache, and the learned-relative attention of one
new token per request over the cached keys.

``run`` computes an operator in plain torch operations when ``own`` is false and through
the package's public binding when it is true. ``exact`` gives the floating-point outputs
in 64 bits, from the definitions.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _decode(name, n, hq, hkv, d, r, w, lo, hi, page, dtype, layout, idle=0, spread=1):
    return dict(name=name, op="decode", n=n, hq=hq, hkv=hkv, d=d, r=r, w=w, len_min=lo, len_max=hi, page=page,
                dtype=dtype, layout=layout, idle=idle, spread=spread)


def _append(name, t, hkv, d, page, dtype, layout, clip, idle=0):
    return dict(name=name, op="append", t=t, hkv=hkv, d=d, page=page, dtype=dtype, layout=layout, clip=clip,
                idle=idle)


def _plan(name, n, page, max_pages, old, new, ended, pad, spread=1):
    return dict(name=name, op="plan", n=n, page=page, max_pages=max_pages, old_max=old, new_max=new, ended=ended,
                pad=pad, spread=spread)


def listed():
    return [
        # one request at the start of its answer, the smallest heads: all latency
        _decode("decode_one_short", 1, 4, 2, 64, 64, 0, 128, 128, 16, "bf16", "nhd"),
        # a local layer of a mixed batch: the window leaves at most 512 keys of each request, three rows are padding
        _decode("decode_local_ragged", 64, 16, 4, 128, 512, 512, 1, 2048, 16, "bf16", "nhd", idle=3),
        # a full layer of a busy server's batch: answers of every length up to 4096
        _decode("decode_batch_ragged", 64, 32, 8, 128, 1024, 0, 16, 4096, 64, "bf16", "nhd"),
        # one user with a long document: few rows, so the work has to be split over the keys
        _decode("decode_long_one", 1, 32, 8, 128, 4096, 0, 32768, 32768, 64, "bf16", "nhd"),
        # several long documents: the largest amount of cache read
        _decode("decode_long_batch", 8, 32, 8, 128, 4096, 0, 32767, 32767, 64, "bf16", "hnd"),
        # long documents kept in 8 bits, eight query heads to a key head, odd lengths
        _decode("decode_long_e4m3", 24, 32, 4, 128, 1024, 0, 8191, 32768, 32, "e4m3", "hnd"),
        # the rows of one decoding step, four of them padding
        _append("append_step", 64, 8, 128, 16, "bf16", "nhd", False, idle=4),
        # a chunk of prompts, keys clipped on the way into the cache
        _append("append_prompt_clip", 32768, 8, 128, 64, "bf16", "nhd", True),
        # an odd number of prompt rows into an 8-bit cache
        _append("append_prompt_e4m3", 16381, 4, 128, 32, "e4m3", "hnd", True, idle=13),
        # one more token for each request of a batch
        _plan("plan_step", 64, 16, 256, 4000, 1, 3, 0),
        # new prompts of every length beside running and ended requests
        _plan("plan_prompts", 256, 64, 128, 4096, 2048, 20, 37),
        # the largest batch: thousands of requests with long tables
        _plan("plan_many", 4096, 16, 512, 8000, 64, 500, 1000),
    ]


def _logint(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("decode", "decode", "append", "plan"))
    page = rng.choice((1, 8, 16, 16, 24, 32, 64, 128))
    dtype = rng.choice(("bf16", "bf16", "e4m3"))
    layout = rng.choice(("nhd", "hnd"))
    if op == "decode":
        hkv = rng.choice((1, 2, 4, 8))
        hq = hkv * rng.choice((1, 2, 3, 4, 5, 8, 8, 16, 20))
        d = rng.choice((64, 128, 128))
        n = _logint(rng, 1, 200)
        # as many cached rows as the largest listed case reads
        most = int(min(32768, 8 * 32767 * 8 * 128 / (n * hkv * d)))
        hi = _logint(rng, 1, most)
        lo = _logint(rng, 1, hi)
        w = rng.choice((0, 0, _logint(rng, 1, 2048)))
        r = 8 * rng.choice((0, 1, 8, 64, 65, 128, 512))
        return dict(op=op, n=n, hq=hq, hkv=hkv, d=d, r=r, w=w, len_min=lo, len_max=hi, page=page, dtype=dtype,
                    layout=layout, idle=rng.choice((0, 0, n // 5)), spread=rng.randrange(1 << 30))
    if op == "append":
        t = _logint(rng, 1, 32768)
        return dict(op=op, t=t, hkv=rng.choice((1, 2, 4, 8)), d=rng.choice((64, 128)), page=page, dtype=dtype,
                    layout=layout, clip=rng.random() < 0.5, idle=rng.choice((0, t // 9)))
    n = _logint(rng, 1, 4096)
    return dict(op=op, n=n, page=page, max_pages=256, old_max=rng.randint(0, 200 * page),
                new_max=max(1, min(_logint(rng, 1, 2048), 56 * page, 200000 // n)), ended=rng.randint(0, n // 4),
                pad=rng.choice((0, rng.randint(0, 3000))), spread=rng.randrange(1 << 30))


# --------------------------------------------------------------------------
# sizes of a case (the same for every seed)
# --------------------------------------------------------------------------
def _lens(c):
    """Cached tokens of each request, the new one among them; 0 for the padding rows at the end."""
    rng = random.Random(c["spread"])
    lens = [_logint(rng, c["len_min"], c["len_max"]) for _ in range(c["n"])]
    lens[0] = c["len_max"]
    for i in range(c["idle"]):
        lens[-1 - i] = 0
    return lens


def _plan_lens(c):
    """(old, new) lengths: running requests grow, new ones start, ended ones drop to 0."""
    rng = random.Random(c["spread"])
    old = [rng.randint(0, c["old_max"]) for _ in range(c["n"])]
    new = [o + rng.randint(min(1, c["new_max"]), c["new_max"]) for o in old]
    for i in rng.sample(range(c["n"]), c["ended"]):
        new[i] = rng.choice((0, old[i] // 2))
    return old, new


def _pages(length, page):
    return -(-length // page)


def _item(c):
    return 2 if c["dtype"] == "bf16" else 1


def work(c):
    if c["op"] == "decode":
        lens = _lens(c)
        seen = [min(x, c["w"]) if c["w"] else x for x in lens]
        keys = sum(seen)
        biased = sum(min(x, c["r"]) for x in seen)
        tables = sum(_pages(x, c["page"]) for x in seen)
        rows = c["n"] * c["hq"]
        return {"bytes": 2 * keys * c["hkv"] * c["d"] * _item(c) + 2 * biased * c["hq"] + 4 * tables + 4 * c["n"]
                + rows * (c["d"] * (2 + 4) + 4 + 4),
                "flops": 4 * keys * c["hq"] * c["d"]}
    if c["op"] == "append":
        live = c["t"] - c["idle"]
        row = c["hkv"] * c["d"]
        return {"bytes": 2 * live * row * (2 + _item(c)) + 8 * c["t"] + (4 * (row + live) if c["clip"] else 0),
                "flops": live * row * (6 if c["clip"] else 1)}
    old, new = _plan_lens(c)
    pages = sum(abs(_pages(b, c["page"]) - _pages(a, c["page"])) for a, b in zip(old, new))
    tokens = sum(max(0, b - a) for a, b in zip(old, new)) + c["pad"]
    return {"bytes": 8 * c["n"] + 8 * pages + 12 * tokens + 8 * c["n"] + 4 + 16, "flops": 0}


# --------------------------------------------------------------------------
# what a program has in hand before the call
# --------------------------------------------------------------------------
def _cache(num_pages, c, gen):
    """A page pool [num_pages, page, hkv, d] (a view of [num_pages, hkv, page, d] for "hnd") and its scales."""
    shape = (num_pages, c["hkv"], c["page"], c["d"]) if c["layout"] == "hnd" else (num_pages, c["page"], c["hkv"], c["d"])
    x = torch.randn(shape, device="cuda", generator=gen)
    scale = None
    if c["dtype"] == "e4m3":
        scale = 0.01 + 0.005 * torch.rand(c["hkv"], device="cuda", generator=gen)
        x.div_(scale.view(1, -1, 1, 1) if c["layout"] == "hnd" else scale.view(1, 1, -1, 1))
        x = x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    else:
        x = x.to(torch.bfloat16)
    return (x.transpose(1, 2) if c["layout"] == "hnd" else x), scale


def _table(lens, page, max_pages, num_pages, gen):
    """A block table [n, max_pages] int32 with pages in random order, -1 behind each request's last, and the pages left."""
    counts = torch.tensor([_pages(x, page) for x in lens], device="cuda")
    first = counts.cumsum(0) - counts
    order = torch.randperm(num_pages, device="cuda", generator=gen).to(torch.int32)
    col = torch.arange(max_pages, device="cuda")
    at = (first[:, None] + col).clamp_(max=num_pages - 1)
    table = torch.where(col < counts[:, None], order[at], -1).to(torch.int32).contiguous()
    return table, order[int(counts.sum()):].contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    s = {"case": c}
    if c["op"] == "decode":
        lens = _lens(c)
        used = sum(_pages(x, c["page"]) for x in lens)
        num_pages = used + used // 8 + 1
        s["k_cache"], s["k_scale"] = _cache(num_pages, c, gen)
        s["v_cache"], s["v_scale"] = _cache(num_pages, c, gen)
        max_pages = _pages(c["len_max"], c["page"])
        s["table"], _ = _table(lens, c["page"], max_pages, num_pages, gen)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = normal(c["n"], c["hq"], c["d"]).to(torch.bfloat16)
        s["profiles"] = (0.5 * normal(c["n"], c["hq"], c["r"])).to(torch.bfloat16) if c["r"] else None
        s["sink"] = normal(c["n"], c["hq"])
    elif c["op"] == "append":
        num_pages = _pages(c["t"], c["page"]) * 5 // 4 + 1
        s["k_cache"], s["k_scale"] = _cache(num_pages, c, gen)
        s["v_cache"], s["v_scale"] = _cache(num_pages, c, gen)
        # the rows of a fused projection: keys and values side by side
        kv = normal(c["t"], 2, c["hkv"], c["d"]).to(torch.bfloat16)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        if c["t"] <= 256:  # a decoding step: every row on a page of its own
            pages = torch.randperm(num_pages * c["page"], device="cuda", generator=gen)[:c["t"]]
            slots = pages
        else:  # prompts: runs of rows on pages in random order
            order = torch.randperm(num_pages, device="cuda", generator=gen)
            i = torch.arange(c["t"], device="cuda")
            slots = order[i // c["page"]] * c["page"] + i % c["page"]
        slots[c["t"] - c["idle"]:] = -1
        s["slots"] = slots.contiguous()
        s["threshold"] = 11.0 if c["d"] == 128 else 8.0
        s["clip_scale"] = 1 + 0.1 * normal(c["hkv"], c["d"]) if c["clip"] else None
        s["tau"] = 1 + 0.1 * normal(c["t"]).abs() if c["clip"] else None
    else:
        old, new = _plan_lens(c)
        used = sum(_pages(x, c["page"]) for x in old)
        grown = sum(max(0, _pages(b, c["page"]) - _pages(a, c["page"])) for a, b in zip(old, new))
        num_pages = used + grown + 16
        s["num_pages"] = num_pages
        s["table"], left = _table(old, c["page"], c["max_pages"], num_pages, gen)
        s["free_pages"] = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
        s["free_pages"][:left.numel()] = left
        s["free_count"] = torch.tensor([left.numel()], dtype=torch.int32, device="cuda")
        s["old"] = torch.tensor(old, dtype=torch.int32, device="cuda")
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        s["max_tokens"] = sum(max(0, b - a) for a, b in zip(old, new)) + c["pad"]
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _plain_decode(s):
    c = s["case"]
    n, hq, hkv, d, r, page = c["n"], c["hq"], c["hkv"], c["d"], c["r"], c["page"]
    num_pages, max_pages = s["k_cache"].shape[0], s["table"].shape[1]
    lens = s["lens"].long()
    span = max_pages * page
    first = torch.zeros_like(lens)
    if c["w"]:
        span = min(span, c["w"])
        first = (lens - c["w"]).clamp(min=0)
    j = first[:, None] + torch.arange(span, device="cuda")
    block = s["table"].long().gather(1, (j // page).clamp(max=max_pages - 1))
    seen = (j < lens[:, None]) & (block >= 0) & (block < num_pages)
    block = block.clamp(0, num_pages - 1)
    keys = s["k_cache"][block, j % page].float()
    values = s["v_cache"][block, j % page].float()
    if s["k_scale"] is not None:
        keys = keys * s["k_scale"][:, None]
        values = values * s["v_scale"][:, None]
    q = s["q"].float().view(n, hkv, hq // hkv, d)
    z = (q @ keys.permute(0, 2, 3, 1)).view(n, hq, span) * d ** -0.5
    if r:
        dist = lens[:, None] - 1 - j
        bias = s["profiles"].float().gather(2, dist.clamp(0, r - 1)[:, None].expand(n, hq, span))
        z = z + torch.where((dist < r)[:, None], bias, 0.0)
    z = torch.where(seen[:, None], z, -math.inf)
    top = torch.maximum(z.amax(2), s["sink"])
    p = torch.exp(z - top[:, :, None])
    total = p.sum(2) + torch.exp(s["sink"] - top)
    out = (p.view(n, hkv, hq // hkv, span) @ values.transpose(1, 2)).view(n, hq, d) / total[:, :, None]
    return {"out": out, "lse": top + torch.log(total)}


def _plain_append(s):
    c = s["case"]
    k, v = s["k"].float(), s["v"].float()
    if c["clip"]:
        z = k * s["clip_scale"]
        norm = z.square().sum(2, keepdim=True).sqrt()
        k = z * (s["threshold"] / norm).clamp(max=1.0) * s["tau"][:, None, None]
        k = k.to(torch.bfloat16).float()
    if c["dtype"] == "e4m3":
        k = (k / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    live = s["slots"] >= 0
    block, row = s["slots"][live] // c["page"], s["slots"][live] % c["page"]
    for cache, x in ((s["k_cache"], k), (s["v_cache"], v)):
        bits = torch.uint8 if c["dtype"] == "e4m3" else torch.int16
        cache.view(bits)[block, row] = x[live].to(cache.dtype).view(bits)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_plan(s):
    c = s["case"]
    n, page, width, room = c["n"], c["page"], c["max_pages"], s["free_pages"].numel()
    old, new = s["old"].long().clamp(0, width * page), s["new"].long().clamp(0, width * page)
    count = s["free_count"].long()
    held, want = (old + page - 1) // page, (new + page - 1) // page
    more, less = (want - held).clamp(min=0), (held - want).clamp(min=0)
    more_at, less_at = more.cumsum(0) - more, less.cumsum(0) - less
    stack_size = count + less.sum()
    taken = torch.minimum(more.sum(), stack_size)
    left = stack_size - taken
    col = torch.arange(width, device="cuda")
    # pages given back go on top of the stack, in the order of the requests
    back = (col >= want[:, None]) & (col < held[:, None])
    spare = room + n * width
    to = torch.where(back, count + less_at[:, None] + col - want[:, None], spare)
    stack = torch.full((spare + 1,), -1, dtype=torch.int32, device="cuda")
    stack[:room] = s["free_pages"]
    stack.scatter_(0, to.view(-1), s["table"].view(-1))
    # and pages taken come from its top
    k = more_at[:, None] + col - held[:, None]
    get = (col >= held[:, None]) & (col < want[:, None])
    page_id = stack[(stack_size - 1 - k).clamp(0, spare)]
    table = torch.where(get, torch.where(k < taken, page_id, s["table"]), s["table"])
    given = torch.minimum((taken - more_at).clamp(min=0), more)
    lens = torch.minimum(new, (held + given) * page)
    fresh = (new - old).clamp(min=0)
    ends = fresh.cumsum(0)
    t = torch.arange(s["max_tokens"], device="cuda")
    who = torch.searchsorted(ends, t, right=True).clamp(max=n - 1)
    real = t < ends[-1]
    pos = old[who] + t - (ends - fresh)[who]
    block = table[who, (pos // page).clamp(0, width - 1)].long()
    held_up = real & (pos < lens[who]) & (block >= 0) & (block < s["num_pages"])
    slots = torch.where(held_up, block * page + pos % page, -1)
    free_pages = torch.where(torch.arange(room, device="cuda") < left, stack[:room], s["free_pages"])
    start = torch.cat([torch.zeros_like(ends[:1]), ends])
    info = torch.cat([left, ends[-1:], more.sum().view(1) - taken, taken])
    return {"block_table": table, "free_pages": free_pages, "lens": lens.to(torch.int32),
            "query_start": start.to(torch.int32), "slots": slots,
            "positions": torch.where(real, pos, 0).to(torch.int32), "info": info.to(torch.int32)}


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"decode": _plain_decode, "append": _plain_append, "plan": _plain_plan}[c["op"]](s)
    from learned_relative_gqa_b200 import binding
    if c["op"] == "decode":
        out, lse = binding.paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["profiles"],
                                        s["sink"], window=c["w"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": out, "lse": lse}
    if c["op"] == "append":
        binding.kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
                          v_scale=s["v_scale"], threshold=s["threshold"] if c["clip"] else None,
                          clip_scale=s["clip_scale"], tau=s["tau"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    p = binding.kv_plan(s["old"], s["new"], s["table"], s["free_pages"], s["free_count"], page_size=c["page"],
                        num_pages=s["num_pages"], max_tokens=s["max_tokens"])
    return {"block_table": s["table"], "free_pages": s["free_pages"], **p}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None
    s = prepare(c, seed)
    if c["op"] == "append":
        rows = {}
        for side in ("k", "v"):
            x = s[side].double()
            if side == "k" and c["clip"]:
                x = x * s["clip_scale"].double()
                length = torch.linalg.vector_norm(x, dim=2, keepdim=True)
                x = torch.where(length > s["threshold"], x * (s["threshold"] / length), x) * s["tau"].double()[:, None, None]
            scale = s[side + "_scale"]
            if scale is not None:
                x = (x / scale.double()[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
            cache = s[side + "_cache"].double()
            at = torch.nonzero(s["slots"] >= 0).view(-1)
            cache[s["slots"][at] // c["page"], s["slots"][at] % c["page"]] = x[at]
            rows[side + "_cache"] = cache
        return rows
    out = torch.zeros(c["n"], c["hq"], c["d"], dtype=torch.float64, device="cuda")
    lse = s["sink"].double().clone()
    group = c["hq"] // c["hkv"]
    for i, length in enumerate(_lens(c)):
        first = max(0, length - c["w"]) if c["w"] else 0
        if length == first:
            continue
        j = torch.arange(first, length, device="cuda")
        block = s["table"][i].long()[j // c["page"]]
        for g in range(c["hkv"]):
            heads = slice(g * group, (g + 1) * group)
            key = s["k_cache"][block, j % c["page"], g].double()
            value = s["v_cache"][block, j % c["page"], g].double()
            if s["k_scale"] is not None:
                key, value = key * s["k_scale"][g].double(), value * s["v_scale"][g].double()
            logits = torch.einsum("hd,jd->hj", s["q"][i, heads].double(), key) / math.sqrt(c["d"])
            near = min(c["r"], length - first)
            if near:  # distance 0 is the last key
                logits[:, logits.shape[1] - near:] += s["profiles"][i, heads, :near].double().flip(1)
            both = torch.logaddexp(torch.logsumexp(logits, 1), s["sink"][i, heads].double())
            out[i, heads] = torch.exp(logits - both[:, None]) @ value
            lse[i, heads] = both
    return {"out": out, "lse": lse}
