"""Workloads of the operators around the paged MXFP4 cache: per-head norm with rotary positions (alone, and in the
pass that writes keys and values into the cache), the pages of the cache (admitting, forking, copying on a write,
freeing, compacting), and attention of sequences that share a long prefix.

Each case runs in two forms on the same inputs.  With ``own`` false the operators are written out in elementary
torch operations, 32 bits wide (angles in 64); with ``own`` true the same work goes through the package's public
functions.  ``exact`` evaluates the definitions in binary64 and is written apart from both.

Rotary positions: a head's first `rot` elements are rot / 2 pairs, pair i turning by position[axis[i]] * inv_freq[i];
a pair is two neighbours (interleaved) or elements i and i + rot / 2 (halves).  The norm, where there is one, comes
first: x / sqrt(mean(x^2) + eps) * weight over the whole head.

MXFP4: 32 consecutive elements of a row share an E8M0 scale 2^(E-127) with E - 127 = floor(log2 max|x|) - 2, and each
element is the nearest E2M1 value (ties to even, saturating at 6) of x / scale; byte j of a row holds element 2j in
its low nibble and 2j+1 in its high one.

Pages: refs counts the rows of the table that hold a page, 0 for a free one.  Token t of row b lies in page
table[b, t // page] at t % page; a row of lens[b] tokens holds its first ceil(lens[b] / page) pages.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_FOUR = 17 / 32  # bytes of one element held in MXFP4: half a byte and 1/32 of a scale
_EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token's queries and keys in a decoding step: latency
        {"name": "rotate token", "op": "rotate", "tokens": 1, "q_heads": 32, "k_heads": 8, "dim": 128, "rot": 128,
         "axes": 1, "pairs": "halves", "norm": True, "far": 100000, "dtype": "bf16"},
        # a vision tower's patches: heads of 80, part of them rotated by row and column, float32
        {"name": "rotate patches fp32", "op": "rotate", "tokens": 1337, "q_heads": 7, "k_heads": 7, "dim": 80,
         "rot": 48, "axes": 2, "pairs": "halves", "norm": False, "far": 512, "dtype": "fp32"},
        # all tokens of a video, normed and rotated by time, height and width: the largest case
        {"name": "rotate video", "op": "rotate", "tokens": 37810, "q_heads": 42, "k_heads": 42, "dim": 128, "rot": 128,
         "axes": 3, "pairs": "neighbours", "norm": True, "far": 512, "dtype": "bf16"},
        # a batch of conversations decodes: queries and keys normed and rotated, keys and values into the cache,
        # attention over it
        {"name": "write and attend batch", "op": "write", "seqs": 192, "shortest": 33, "longest": 1025, "queries": 1,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "axes": 1, "pairs": "halves", "norm": True, "page": 64,
         "dtype": "bf16"},
        # three prompts with pictures in them are taken in by a chunk: positions of three axes
        {"name": "write and attend chunk", "op": "write", "seqs": 3, "shortest": 1000, "longest": 4099, "queries": 500,
         "q_heads": 16, "kv_heads": 4, "dim": 64, "rot": 48, "axes": 3, "pairs": "halves", "norm": True, "page": 16,
         "dtype": "fp16"},
        # parallel samples: 12 prompts fork into 5 rows each, whose next token copies the shared last page
        {"name": "fork samples", "op": "fork", "parents": 12, "children": 5, "shortest": 65, "longest": 8190,
         "kv_heads": 8, "dim": 128, "page": 64, "spare": 300},
        # prompts come into a large pool of small pages, most of which is taken
        {"name": "admit prompts", "op": "admit", "rows": 256, "live": 200, "shortest": 17, "longest": 16385,
         "kv_heads": 1, "dim": 64, "page": 16, "spare": 40000},
        # a cache in which conversations have come and gone is made compact
        {"name": "compact cache", "op": "compact", "rows": 160, "shortest": 130, "longest": 4097, "kv_heads": 8,
         "dim": 128, "page": 64, "spare": 3000},
        # a few samples of one prompt decode: latency
        {"name": "shared samples", "op": "shared", "groups": 1, "seqs": 4, "prefix": 2049, "suffix": 300,
         "queries": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # two system prompts, each shared by a batch of conversations of ragged lengths
        {"name": "shared prompts", "op": "shared", "groups": 2, "seqs": 32, "prefix": 16001, "suffix": 1025,
         "queries": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
        # drafts of several tokens are checked against shared documents, small pages
        {"name": "shared drafts", "op": "shared", "groups": 5, "seqs": 7, "prefix": 5003, "suffix": 257,
         "queries": 6, "q_heads": 16, "kv_heads": 4, "dim": 64, "page": 16, "dtype": "fp16"},
        # many requests on one long document
        {"name": "shared document", "op": "shared", "groups": 1, "seqs": 128, "prefix": 32769, "suffix": 2001,
         "queries": 1, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "write", "fork", "admit", "compact", "shared", "shared", "shared"])
    axes, pairs = rng.choice([1, 2, 3]), rng.choice(["halves", "neighbours"])
    if op == "rotate":
        dim = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        q_heads = _log(rng, 1, 64)
        k_heads = rng.choice([0, 1, q_heads, max(1, q_heads // 4)])
        return {"op": op, "tokens": _log(rng, 1, max(1, 150_000_000 // ((q_heads + k_heads) * dim))),
                "q_heads": q_heads, "k_heads": k_heads, "dim": dim, "rot": rng.choice([dim, 16 * rng.randint(1, dim // 16)]),
                "axes": axes, "pairs": pairs, "norm": rng.random() < 0.7, "far": _log(rng, 16, 1_000_000),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 7, 8])
    dim, page = rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "write":
        longest = _log(rng, 2, 8192)
        queries = 1 if rng.random() < 0.6 else _log(rng, 2, min(512, longest))
        cost = max(longest * kv_heads * dim * 2, longest * kv_heads * group * queries)
        return {"op": op, "seqs": _log(rng, 1, max(1, min(256, 500_000_000 // cost))),
                "shortest": _log(rng, queries, longest), "longest": longest, "queries": queries,
                "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([dim, 16 * rng.randint(1, dim // 16)]), "axes": axes, "pairs": pairs,
                "norm": rng.random() < 0.7, "page": page, "dtype": dtype}
    if op == "fork":
        longest = _log(rng, 2, 16384)
        return {"op": op, "parents": _log(rng, 1, max(1, min(64, 300_000 // longest))), "children": rng.randint(1, 9),
                "shortest": _log(rng, 1, longest), "longest": longest, "kv_heads": kv_heads, "dim": dim, "page": page,
                "spare": _log(rng, 700, 5000)}
    if op == "admit":
        rows = _log(rng, 2, 512)
        longest = _log(rng, 2, max(2, min(32768, 2_000_000 // rows)))
        return {"op": op, "rows": rows, "live": rng.randint(1, rows - 1), "shortest": _log(rng, 1, longest),
                "longest": longest, "kv_heads": 1, "dim": 64, "page": page, "spare": rows * (longest // page + 2)}
    if op == "compact":
        longest = _log(rng, 2, 8192)
        return {"op": op, "rows": _log(rng, 1, max(1, min(256, 400_000 // longest))), "shortest": _log(rng, 1, longest),
                "longest": longest, "kv_heads": kv_heads, "dim": dim, "page": page, "spare": _log(rng, 10, 4000)}
    queries = 1 if rng.random() < 0.6 else _log(rng, 2, 64)
    prefix, suffix = _log(rng, 1, 32768), _log(rng, queries, 4096)
    cost = max(kv_heads * group * queries * prefix, (suffix + 2 * page) * kv_heads * dim * 2,
               kv_heads * group * queries * (suffix + 2 * page))
    seqs = _log(rng, 1, max(1, min(64, 250_000_000 // cost)))
    groups = _log(rng, 1, max(1, min(6, 250_000_000 // (cost * seqs), 250_000_000 // (prefix * kv_heads * dim * 2))))
    return {"op": op, "groups": groups, "seqs": seqs, "prefix": prefix, "suffix": suffix, "queries": queries,
            "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype}


def _spread(n, lo, hi):
    """n lengths from `hi` down to `lo` in equal ratios."""
    return [hi] if n == 1 else [int(round(hi * (lo / hi) ** (b / (n - 1)))) for b in range(n)]


def _new_tokens(case, lens):
    """New tokens of each sequence of a "write" case: all alike for one, else falling along the batch."""
    n = case["seqs"]
    return [min(lens[b], max(1, case["queries"] * (n - b) // n)) for b in range(n)]


def _shared_sizes(case):
    """(first sequence of each group and their number, tokens in common by group, lengths, queries).

    Groups grow smaller and their prefixes shorter; a sequence has from `queries` to `suffix` tokens of its own."""
    starts, shared, lens, new = [0], [], [], []
    for g in range(case["groups"]):
        n = max(1, case["seqs"] * (case["groups"] - g) // case["groups"])
        p = max(1, case["prefix"] - g * (case["prefix"] // (2 * case["groups"])))
        starts.append(starts[-1] + n)
        shared.append(p)
        own_tokens = _spread(n, case["queries"], max(case["queries"], case["suffix"] - g))
        lens += [p + t for t in own_tokens]
        new += [max(1, case["queries"] - (b % 3 if case["queries"] > 3 else 0)) for b in range(n)]
    return starts, shared, lens, new


def _page_bytes(case):
    return 2 * case["kv_heads"] * case["page"] * case["dim"] * _FOUR


def _pool(case):
    """Lengths of the rows, and the pages in use and in the pool, of a case of page operations."""
    page = case["page"]
    if case["op"] == "fork":
        lens = _spread(case["parents"], case["shortest"], case["longest"])
        rows = lens + [0] * (case["parents"] * case["children"])
    elif case["op"] == "admit":
        lens = _spread(case["rows"], case["shortest"], case["longest"])
        rows = [n if i % case["rows"] < case["live"] else 0 for i, n in enumerate(lens[::-1])]
    else:
        rows = _spread(case["rows"], case["shortest"], case["longest"])
    used = sum(-(-n // page) for n in rows)
    return rows, used, used + case["spare"]


def work(case):
    op = case["op"]
    if op == "rotate":
        s, heads = _BYTES[case["dtype"]], case["q_heads"] + case["k_heads"]
        return {"bytes": case["tokens"] * (2 * heads * case["dim"] * s + 4 * case["axes"]), "flops": 0}
    if op == "write":
        s, d, hq, hkv = _BYTES[case["dtype"]], case["dim"], case["q_heads"], case["kv_heads"]
        lens = _spread(case["seqs"], case["shortest"], case["longest"])
        new = _new_tokens(case, lens)
        tokens = sum(new)
        pairs = sum(n * (length - n) + n * (n + 1) // 2 for length, n in zip(lens, new))
        old = sum(lens) - tokens
        return {"bytes": tokens * d * (s * (3 * hq + 2 * hkv) + 2 * hkv * _FOUR) + 2 * old * hkv * d * _FOUR,
                "flops": 4 * pairs * hq * d}
    if op in ("fork", "admit", "compact"):
        rows, used, pool = _pool(case)
        page, held = case["page"], sum(1 for n in rows if n)
        if op == "fork":  # the children's rows are written; a page is copied for each whose last one is not full
            entries = sum(-(-n // page) * (1 + case["children"]) for n in rows[:case["parents"]])
            copied = sum(case["children"] for n in rows[:case["parents"]] if n % page)
            return {"bytes": 4 * entries + 8 * pool + 2 * copied * _page_bytes(case) + 24 * len(rows), "flops": 0}
        if op == "admit":  # a slot for each token, a table entry for each page
            lens = _spread(case["rows"], case["shortest"], case["longest"])[::-1][case["live"]:]
            return {"bytes": 8 * sum(lens) + 8 * sum(-(-n // page) for n in lens) + 8 * pool + 24 * len(rows),
                    "flops": 0}
        moved = used * (pool - used) // pool  # of pages in random places
        return {"bytes": 2 * moved * _page_bytes(case) + 12 * pool + 8 * used + 8 * held, "flops": 0}
    s, d, hq, hkv = _BYTES[case["dtype"]], case["dim"], case["q_heads"], case["kv_heads"]
    starts, shared, lens, new = _shared_sizes(case)
    keys, pairs = sum(shared), 0
    for g, p in enumerate(shared):
        for b in range(starts[g], starts[g + 1]):
            keys += lens[b] - p
            pairs += new[b] * (lens[b] - new[b]) + new[b] * (new[b] + 1) // 2
    return {"bytes": 2 * keys * hkv * d * _FOUR + 2 * sum(new) * hq * d * s, "flops": 4 * pairs * hq * d}


# ------------------------------------------- MXFP4 in elementary operations --

def _power(e):
    """2^(e - 127) in float32 for whole e in 0..254, from its bits."""
    e = e.to(torch.int32)
    return torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _encode(x):
    """float32 [..., 32 b] -> packed E2M1 codes [..., 16 b] and E8M0 codes [..., b]."""
    blocks = x.unflatten(-1, (-1, 32))
    amax = blocks.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    y = (blocks * _power(127 - e).unsqueeze(-1)).abs()
    code = torch.signbit(blocks).to(torch.uint8) * 8
    code += (y > 0.25).to(torch.uint8) + (y >= 0.75).to(torch.uint8) + (y > 1.25).to(torch.uint8)
    code += (y >= 1.75).to(torch.uint8) + (y > 2.5).to(torch.uint8) + (y >= 3.5).to(torch.uint8)
    code += (y > 5.0).to(torch.uint8)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _decode(packed, scales):
    """Packed codes [..., d/2] and E8M0 codes [..., d/32] -> float32 [..., d]."""
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).to(torch.int32)
    two = code & 7  # 0 .5 1 1.5 2 3 4 6
    mag = torch.where(two < 4, two.float() * 0.5, torch.where(two < 6, two.float() - 2.0, two.float() * 2.0 - 8.0))
    val = torch.where(code >= 8, -mag, mag)
    return (val.reshape(*scales.shape, 32) * _power(scales).unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------ inputs --

def _rotary(case):
    """(inv_freq float64 [pairs], axis int32 [pairs], turns int64 [pairs]): frequencies of each axis' own section for
    neighbours, of the whole for halves; turns are inv_freq / 2 pi in units of 2^-64 turn, wrapping around."""
    pairs, axes = case["rot"] // 2, case["axes"]
    i = torch.arange(pairs, dtype=torch.float64)
    axis = (i * axes / pairs).floor().to(torch.int32)  # sections of (nearly) equal size
    if case["pairs"] == "neighbours":
        first = torch.tensor([(axis == a).nonzero().min() if (axis == a).any() else 0 for a in range(axes)])
        size = torch.tensor([max(1, int((axis == a).sum())) for a in range(axes)])
        expo = (i - first[axis.long()]) / size[axis.long()]
    else:
        expo = i / pairs
    inv_freq = 10000.0 ** -expo
    t = inv_freq / (2 * math.pi) * 2.0 ** 32
    turns = (t.floor().to(torch.int64) << 32) + ((t - t.floor()) * 2.0 ** 32).round().to(torch.int64)
    return inv_freq.cuda(), axis.cuda(), turns.cuda()


def _rows(shape, g, dt):
    """Projected heads: most channels near 1, a few large."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., ::17] *= 4.0
    return x.to(dt)


def _weights(case, g, dt):
    if not case["norm"]:
        return None, None
    w = 1.0 + 0.2 * torch.randn(2, case["dim"], generator=g, device="cuda")
    return w[0].to(dt), w[1].to(dt)


def _cache(g, pages, heads, page, d):
    """Codes and scales of a cache of random tokens; keys have a few large channels."""
    chan = torch.ones(heads, 1, d, device="cuda")
    chan[..., ::17] = 6.0
    state = {}
    for name in ("k", "v"):
        x = torch.randn((pages, heads, page, d), generator=g, device="cuda")
        state[name + "_codes"], state[name + "_scales"] = _encode(x * chan if name == "k" else x)
    return state


def _byte_cache(case, g, pages):
    """A cache of arbitrary bytes, for what only moves them."""
    shape = (pages, case["kv_heads"], case["page"])
    return {name: torch.randint(0, 255, (*shape, case["dim"] // (2 if "codes" in name else 32)), generator=g,
                                device="cuda", dtype=torch.uint8) for name in _CACHE}


_CACHE = ("k_codes", "k_scales", "v_codes", "v_scales")


def _deal(order, counts):
    """A block table [rows, most + 1] that takes the pages of `order` row by row; places behind a row's are 0."""
    table = torch.zeros(len(counts), max(counts) + 1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table


def _int(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op in ("rotate", "write"):
        dt = _DTYPES[case["dtype"]]
        state["inv_freq"], state["axis"], state["turns"] = _rotary(case)
    if op == "rotate":
        n, hq, hk, axes = case["tokens"], case["q_heads"], case["k_heads"], case["axes"]
        x = _rows((n, hq + 2 * hk, case["dim"]), g, dt)  # the projection's output: queries, keys, values
        t = torch.arange(n, device="cuda")
        side = max(1, math.isqrt(max(1, n // 10)))
        grid = (t,) if axes == 1 else (t // side, t % side) if axes == 2 else (t // (side * side), t // side % side, t % side)
        first = torch.randint(-case["far"] // 4, case["far"], (axes,), generator=g, device="cuda")
        state["positions"] = (torch.stack(grid, 1) + first).to(torch.int32)
        state["q"], state["k"] = x[:, :hq], x[:, hq:hq + hk] if hk else None
        state["q_weight"], state["k_weight"] = _weights(case, g, dt)
        return state
    page, d, heads = case["page"], case["dim"], case["kv_heads"]
    if op == "write":
        lens = _spread(case["seqs"], case["shortest"], case["longest"])
        new = _new_tokens(case, lens)
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        state["table"] = _deal(order, counts)
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).cuda()
        pos = torch.cat([torch.arange(length - n, length) for length, n in zip(lens, new)]).cuda()
        state["slots"] = state["table"][seq, pos // page].long() * page + pos % page
        state |= _cache(g, pages, heads, page, d)
        x = _rows((len(pos), case["q_heads"] + 2 * heads, d), g, dt)
        state["q"], state["k"], state["v"] = x.split((case["q_heads"], heads, heads), 1)
        axes = case["axes"]
        state["positions"] = (pos.unsqueeze(1) // torch.tensor([1, 3, 7]).cuda()[:axes]).to(torch.int32)
        state["q_weight"], state["k_weight"] = _weights(case, g, dt)
        state["lens"], state["most"] = _int(lens), max(new)
        state["q_starts"] = _int([0] + new).cumsum(0).to(torch.int32)
        return state
    if op in ("fork", "admit", "compact"):
        rows, used, pages = _pool(case)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        counts = [-(-n // page) for n in rows]
        table = _deal(order, counts)
        refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        refs[order[:used].long()] = 1
        if op == "fork":
            wide = max(counts) + 1
            table = torch.nn.functional.pad(table, (0, wide - table.shape[1]))
            kids = [b for b in range(case["parents"]) for _ in range(case["children"])]
            mine = list(range(case["parents"]))
            state["fork"] = _int(mine + kids)
            state["back"] = _int(mine + [-1] * len(kids))
            state["counts"] = _int([0] * case["parents"] + [1] * len(kids))
            state["total"] = len(kids)
        elif op == "admit":
            lens = _spread(case["rows"], case["shortest"], case["longest"])[::-1]
            most = max(-(-n // page) for n in lens)
            table = torch.nn.functional.pad(table, (0, max(0, most - table.shape[1])))
            grow = [0 if n else lens[i] for i, n in enumerate(rows)]
            state["back"] = _int([i if n else -1 for i, n in enumerate(rows)])
            state["counts"], state["total"] = _int(grow), sum(grow)
        else:
            # half of the rows share the first pages of the row before them
            both = torch.arange(1, len(rows), 2)
            for b in both.tolist():
                n = min(counts[b], counts[b - 1]) // 2
                refs[table[b, :n].long()] -= 1
                table[b, :n] = table[b - 1, :n]
                refs[table[b, :n].long()] += 1
            state["table0"], state["refs0"] = table.clone(), refs.clone()
        state |= _byte_cache(case, g, pages)
        state |= {"table": table.contiguous(), "refs": refs, "lens": _int(rows)}
        return state
    dt = _DTYPES[case["dtype"]]
    starts, shared, lens, new = _shared_sizes(case)
    counts, fresh = [-(-n // page) for n in lens], []  # pages of each row, and those that are its own
    for k, p in enumerate(shared):
        fresh += [counts[b] if b == starts[k] else counts[b] - p // page for b in range(starts[k], starts[k + 1])]
    pages = sum(fresh) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(counts) + 1, dtype=torch.int32, device="cuda")
    at = 0
    for k, p in enumerate(shared):
        for b in range(starts[k], starts[k + 1]):
            table[b, counts[b] - fresh[b]:counts[b]] = order[at:at + fresh[b]]
            at += fresh[b]
            if b > starts[k]:
                table[b, :p // page] = table[starts[k], :p // page]
    state |= _cache(g, pages, heads, page, d)
    for k, p in enumerate(shared):  # the page that the prefix ends in is a copy for each
        if p % page:
            first = int(table[starts[k], p // page])
            others = table[starts[k] + 1:starts[k + 1], p // page].long()
            for name in _CACHE:
                state[name][others, :, :p % page] = state[name][first, :, :p % page]
    state |= {"table": table, "lens": _int(lens), "groups": _int(starts), "shared": _int(shared),
              "q": torch.randn((sum(new), case["q_heads"], d), generator=g, device="cuda").to(dt),
              "q_starts": _int([0] + new).cumsum(0).to(torch.int32), "most": max(new),
              "most_group": max(sum(new[a:b]) for a, b in zip(starts, starts[1:]))}
    return state


# -------------------------------------------------------------- plain forms --

def _plain_rotate(s, x, weight):
    """Norm and rotation of x [tokens, heads, dim] in float32."""
    case = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * weight.float()
    turn = s["positions"].double()[:, s["axis"].long()] * s["inv_freq"]
    c, n = turn.cos().float().unsqueeze(1), turn.sin().float().unsqueeze(1)
    rot = case["rot"]
    if case["pairs"] == "neighbours":
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _parts(q, k, v, seen):
    """softmax numerators: q [b, heads, rows, d], k and v [b, heads, tokens, d], seen broadcast to [b, heads, rows,
    tokens].  (top score [..., 1], sum, weighted values) of the keys that a row sees."""
    scores = ((q @ k.transpose(2, 3)) * q.shape[-1] ** -0.5).masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    weight = (scores - top).exp_()
    return top, weight.sum(-1, keepdim=True), weight @ v


def _padded_queries(q, starts, most, heads):
    """Rows starts[b] .. starts[b + 1] of q as [b, heads, group * most, d] float32, and [b, most] whether there is one."""
    n = (starts[1:] - starts[:-1]).unsqueeze(1)
    i = torch.arange(most, device="cuda")
    rows = (starts[:-1].unsqueeze(1) + i).clamp(max=len(q) - 1).long()
    x = q.float()[rows].unflatten(2, (heads, -1)).permute(0, 2, 3, 1, 4)  # [b, heads, group, most, d]
    return x.flatten(2, 3), i < n


def _rows_back(x, real, most):
    """The inverse, of [b, heads, group * most, w]: [rows, heads * group, w]."""
    return x.unflatten(2, (-1, most)).permute(0, 3, 1, 2, 4).flatten(2, 3)[real]


def _keys(s, name, table, lens):
    """float32 [b, heads, tokens, d] of the tables' pages, zeros past the lengths."""
    table = table.long()
    x = _decode(s[name + "_codes"][table], s[name + "_scales"][table]).transpose(1, 2).flatten(2, 3)
    return x.masked_fill((torch.arange(x.shape[2], device="cuda") >= lens.unsqueeze(1))[:, None, :, None], 0.0)


def _plain_attend(s, q):
    case = s["case"]
    x, real = _padded_queries(q, s["q_starts"], s["most"], case["kv_heads"])
    k, v = _keys(s, "k", s["table"], s["lens"]), _keys(s, "v", s["table"], s["lens"])
    n = s["q_starts"][1:] - s["q_starts"][:-1]
    p = (s["lens"] - n).unsqueeze(1) + torch.arange(s["most"], device="cuda")
    seen = torch.arange(k.shape[2], device="cuda") <= p.unsqueeze(2)
    _, total, out = _parts(x, k, v, seen.repeat(1, case["q_heads"] // case["kv_heads"], 1).unsqueeze(1))
    return _rows_back(out / total.clamp(min=1e-37), real, s["most"]).to(q.dtype)


def _plain_write(s):
    q = _plain_rotate(s, s["q"], s["q_weight"]).to(s["q"].dtype)
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    for name, x in (("k", _plain_rotate(s, s["k"], s["k_weight"])), ("v", s["v"].float())):
        s[name + "_codes"][at, :, off], s[name + "_scales"][at, :, off] = _encode(x)
    return {"q": q, "out": _plain_attend(s, q)}


def _plain_shared(s):
    """The prefix of each group once for all its queries, then every sequence's own tokens, and both joined."""
    case = s["case"]
    page, heads, group = case["page"], case["kv_heads"], case["q_heads"] // case["kv_heads"]
    firsts = s["groups"][:-1].long()
    x, real = _padded_queries(s["q"], s["q_starts"][s["groups"].long()], s["most_group"], heads)
    columns = -(-case["prefix"] // page)
    k, v = (_keys(s, name, s["table"][firsts, :columns], s["shared"]) for name in ("k", "v"))
    seen = (torch.arange(k.shape[2], device="cuda") < s["shared"].unsqueeze(1))[:, None, None]
    first = [_rows_back(t, real, s["most_group"]) for t in _parts(x, k, v, seen)]
    # own tokens: from the page that the prefix ends in
    which = torch.searchsorted(s["groups"][1:], torch.arange(len(s["lens"]), device="cuda", dtype=torch.int32), right=True)
    shared = s["shared"][which]
    x, real = _padded_queries(s["q"], s["q_starts"], s["most"], heads)
    column = (shared // page).unsqueeze(1) + torch.arange((case["suffix"] + page - 1) // page + 1, device="cuda")
    table = s["table"].gather(1, column.clamp(max=s["table"].shape[1] - 1).long())
    skip = shared // page * page
    k, v = (_keys(s, name, table, s["lens"] - skip) for name in ("k", "v"))
    n = s["q_starts"][1:] - s["q_starts"][:-1]
    p = (s["lens"] - n).unsqueeze(1) + torch.arange(s["most"], device="cuda")
    j = skip.unsqueeze(1) + torch.arange(k.shape[2], device="cuda")
    seen = (j.unsqueeze(1) <= p.unsqueeze(2)) & (j >= shared.unsqueeze(1)).unsqueeze(1)
    second = [_rows_back(t, real, s["most"]) for t in _parts(x, k, v, seen.repeat(1, group, 1).unsqueeze(1))]
    top = torch.maximum(first[0], second[0])
    a, b = (first[0] - top).exp(), (second[0] - top).exp()
    return ((first[2] * a + second[2] * b) / (first[1] * a + second[1] * b)).to(s["q"].dtype)


def _held(lens, page):
    return torch.div(lens + page - 1, page, rounding_mode="floor")


def _plain_select(s, sources):
    """Every row becomes what row sources[b] was (-1: empty)."""
    page, table, refs = s["case"]["page"], s["table"], s["refs"]
    old = s["lens"]
    new = torch.where(sources >= 0, old[sources.clamp(min=0).long()], 0)
    column = torch.arange(table.shape[1], device="cuda")
    had, has = (column < _held(n, page).unsqueeze(1) for n in (old, new))
    taken = torch.where(has, table[sources.clamp(min=0).long()], table)
    refs.index_add_(0, table.flatten().long(), -had.flatten().to(torch.int32))
    refs.index_add_(0, taken.flatten().long(), has.flatten().to(torch.int32))
    table.copy_(taken)
    old.copy_(new)


def _plain_extend(s, counts, total):
    """Pages for counts[b] more tokens of every row: (slots of the new tokens, pages to copy [rows, 2], pages short)."""
    page, table, refs, lens = s["case"]["page"], s["table"], s["refs"], s["lens"]
    rows, pages = len(lens), len(refs)
    b = torch.arange(rows, device="cuda")
    at = (lens // page).clamp(max=table.shape[1] - 1).long()
    last = table[b, at].long()
    into = (counts > 0) & (lens % page > 0)  # the next token goes into a page that has some
    last = torch.where(into, last, pages)
    writers = torch.zeros(pages + 1, dtype=torch.int32, device="cuda").index_add_(0, last, torch.ones_like(lens))
    lowest = torch.full((pages + 1,), rows, device="cuda").scatter_reduce_(0, last, b, "amin")
    owners = torch.cat((refs, refs.new_ones(1)))[last]
    copy = into & ~((writers[last] == owners) & (lowest[last] == b))
    have, want = _held(lens, page), _held(lens + counts, page)
    need = want - have + copy
    after = need.cumsum(0)
    before = (after - need).long()
    free = refs == 0
    rank = free.cumsum(0)
    short = (after[-1] - rank[-1]).clamp(min=0)
    ok = short == 0
    pool = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    pool[torch.where(free, rank - 1, pages)] = torch.arange(pages, dtype=torch.int32, device="cuda")
    column = torch.arange(table.shape[1], device="cuda")
    copies = torch.stack((last.to(torch.int32), pool[before.clamp(max=pages)]), 1)
    copies = torch.where((copy & ok).unsqueeze(1), copies, -1)
    fresh = (column >= have.unsqueeze(1)) & (column < want.unsqueeze(1))
    index = (before + copy).unsqueeze(1) + column - have.unsqueeze(1)
    grown = torch.where(fresh, pool[index.clamp(0, pages)], table)
    grown = torch.where(copy.unsqueeze(1) & (column == at.unsqueeze(1)), copies[:, 1:], grown)
    table.copy_(torch.where(ok, grown, table))
    taken = free & (rank <= after[-1])
    leave = torch.zeros(pages + 1, dtype=torch.int32, device="cuda").index_add_(0, last, copy.to(torch.int32))[:pages]
    refs.copy_(torch.where(ok, torch.where(taken, 1, refs - leave), refs))
    upto = counts.cumsum(0)
    i = torch.arange(total, device="cuda")
    row = torch.searchsorted(upto, i, right=True).clamp(max=rows - 1)
    t = lens[row] + i - (upto - counts)[row]
    slots = table[row, (t // page).clamp(max=table.shape[1] - 1).long()].long() * page + t % page
    lens.copy_(torch.where(ok, lens + counts, lens))
    return torch.where(ok, slots, -1), copies, short.to(torch.int32).reshape(1)


def _plain_compact(s):
    """Pages at `used` and above go to free places below it: (moves [pages // 2, 2], used)."""
    page, table, refs = s["case"]["page"], s["table"], s["refs"]
    pages = len(refs)
    idx = torch.arange(pages, device="cuda")
    held = refs > 0
    used = held.sum()
    hole, mover = ~held & (idx < used), held & (idx >= used)
    size = pages // 2
    moves = torch.full((size + 1, 2), -1, dtype=torch.int32, device="cuda")
    for at, which in ((0, mover), (1, hole)):
        moves[torch.where(which, which.cumsum(0) - 1, size), at] = idx.to(torch.int32)
    moves[size] = -1
    moves = moves[:size]
    to = idx.clone().to(torch.int32)
    real = moves[:, 0] >= 0
    to = torch.cat((to, to.new_zeros(1)))
    to[torch.where(real, moves[:, 0], pages).long()] = moves[:, 1]
    column = torch.arange(table.shape[1], device="cuda")
    table.copy_(torch.where(column < _held(s["lens"], page).unsqueeze(1), to[table.long()], table))
    moved = torch.zeros_like(refs).index_add_(0, to[:pages].long(), refs)
    refs.copy_(moved)
    return moves, used.to(torch.int32).reshape(1)


def _plain_copy(s, pairs):
    src, dst = pairs[pairs[:, 0] >= 0].long().unbind(1)
    for name in _CACHE:
        s[name][dst] = s[name][src]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(state)
    if op == "rotate":
        return [_plain_rotate(state, state[n], state[n + "_weight"]).to(state[n].dtype)
                for n in ("q", "k") if state[n] is not None]
    if op == "write":
        return _plain_write(state)
    if op == "shared":
        return _plain_shared(state)
    if op == "compact":
        state["table"].copy_(state["table0"])
        state["refs"].copy_(state["refs0"])
        moves, used = _plain_compact(state)
        _plain_copy(state, moves)
        out = {"moves": moves, "used": used}
    else:
        if op == "fork":
            _plain_select(state, state["fork"])
        slots, copies, short = _plain_extend(state, state["counts"], state["total"])
        if op == "fork":
            _plain_copy(state, copies)
        _plain_select(state, state["back"])
        out = {"slots": slots, "copies": copies, "short": short}
    return out | {n: state[n] for n in ("table", "refs", "lens") + (_CACHE if op != "admit" else ())}


def _run_own(state):
    import diffusion_transformer_mlp_gb300 as fc2
    case = state["case"]
    op = case["op"]
    if op in ("rotate", "write"):
        rotary = fc2.HeadRotary(state["turns"], state["axis"], case["pairs"] == "neighbours")
        if op == "rotate":
            out = fc2.head_norm_rotary(state["q"], state["k"], rotary, state["positions"], state["q_weight"],
                                       None if state["k"] is None else state["k_weight"], _EPS)
            return [t for t in out if t is not None]
    if op != "rotate":
        cache = fc2.MXFP4Cache(*(state[n] for n in _CACHE)) if op != "admit" else None
    if op == "write":
        q = fc2.mxfp4_cache_write_rotary(cache, state["q"], state["k"], state["v"], state["slots"], rotary,
                                         state["positions"], state["q_weight"], state["k_weight"], _EPS)
        return {"q": q, "out": fc2.mxfp4_cache_attention(q, cache, state["table"], state["lens"], state["q_starts"],
                                                         state["most"])}
    if op == "shared":
        return fc2.mxfp4_cache_attention_shared(state["q"], cache, state["table"], state["lens"], state["groups"],
                                                state["shared"], state["q_starts"], state["most"],
                                                state["most_group"])
    if op == "compact":
        state["table"].copy_(state["table0"])
        state["refs"].copy_(state["refs0"])
    pages = fc2.MXFP4Pages(state["refs"], state["table"], state["lens"], case["page"])
    if op == "compact":
        moves, used = fc2.mxfp4_pages_compact(pages)
        fc2.mxfp4_cache_copy(cache, moves)
        out = {"moves": moves, "used": used}
    else:
        if op == "fork":
            fc2.mxfp4_pages_select(pages, state["fork"])
        slots, copies, short = fc2.mxfp4_pages_extend(pages, state["counts"], state["total"])
        if op == "fork":
            fc2.mxfp4_cache_copy(cache, copies)
        fc2.mxfp4_pages_select(pages, state["back"])
        out = {"slots": slots, "copies": copies, "short": short}
    return out | {n: state[n] for n in ("table", "refs", "lens") + (_CACHE if op != "admit" else ())}


# ----------------------------------------------------- definitions, binary64 --

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_power(e):
    """2^e in binary64 for whole e, from its bits (pow on the GPU is off by an ulp for some)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(x):
    """What MXFP4 holds of the rows of x: the quantum of the E2M1 grid at |y| is 1/2 below 2, 1 below 4 and 2 above,
    and torch.round takes ties to even multiples of it, which are the even codes."""
    b = x.double().unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -125)
    one = torch.floor(torch.log2(a))  # off by one where log2 rounds up to a whole number: put right below
    one = torch.where(_exact_power(one) > a, one - 1, torch.where(_exact_power(one + 1) <= a, one + 1, one))
    y = b.abs() / _exact_power(one - 2)
    quantum = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    y = (torch.round(y / quantum) * quantum).clamp(max=6.0)
    return (torch.copysign(y, b) * _exact_power(one - 2)).flatten(-2)


def _exact_decode(packed, scales):
    """float64 values of packed codes [..., d/2] with E8M0 codes [..., d/32]."""
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float64, device=packed.device)
    x = torch.stack((grid[(packed % 16).long()], grid[(packed // 16).long()]), -1).reshape(*packed.shape[:-1], -1)
    return x * _exact_power(scales.long() - 127).repeat_interleave(32, -1)


def _exact_rotate(s, x, weight):
    """Norm and rotation in binary64, a pair as a complex number."""
    case = s["case"]
    y = x.double()
    if weight is not None:
        y = y / (y.square().sum(-1, keepdim=True) / y.shape[-1] + _EPS).sqrt() * weight.double()
    half = case["rot"] // 2
    pairs = torch.arange(case["rot"], device="cuda").reshape(half, 2) if case["pairs"] == "neighbours" else \
        torch.arange(case["rot"], device="cuda").reshape(2, half).T
    angle = torch.stack([s["positions"][:, int(a)].double() * f for a, f in zip(s["axis"].tolist(), s["inv_freq"])], 1)
    z = torch.complex(y[..., pairs[:, 0]], y[..., pairs[:, 1]]) * torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    y = y.clone()
    y[..., pairs[:, 0]], y[..., pairs[:, 1]] = z.real, z.imag
    return y


def _exact_attend(s, q, lens, starts, fresh=None):
    """Attention row by row; `fresh` are the values of new keys and values at the ends of the sequences."""
    case = s["case"]
    page, hkv, d, outs = case["page"], case["kv_heads"], case["dim"], []
    for b, length in enumerate(lens):
        n = starts[b + 1] - starts[b]
        pages = s["table"][b, :-(-length // page)].long()
        kv = []
        for i, name in enumerate(("k", "v")):
            x = _exact_decode(s[name + "_codes"][pages], s[name + "_scales"][pages]).transpose(1, 2).flatten(0, 1)[:length]
            if fresh is not None:
                x = torch.cat((x[:length - n], fresh[i][starts[b]:starts[b + 1]]))
            kv.append(x.transpose(0, 1))  # [heads, tokens, d]
        qb = q[starts[b]:starts[b + 1]].double().unflatten(1, (hkv, -1)).permute(1, 2, 0, 3)  # [heads, group, n, d]
        scores = qb @ kv[0].transpose(1, 2).unsqueeze(1) / math.sqrt(d)
        hide = torch.arange(length, device="cuda") > torch.arange(length - n, length, device="cuda").unsqueeze(1)
        o = torch.softmax(scores.masked_fill(hide, -math.inf), -1) @ kv[1].unsqueeze(1)
        outs.append(o.permute(2, 0, 1, 3).flatten(1, 2))
    return torch.cat(outs)


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "admit", "compact"):
        return None  # whole numbers and bytes
    s = prepare(case, seed)
    if op == "rotate":
        return [_exact_rotate(s, s[n], s[n + "_weight"]) for n in ("q", "k") if s[n] is not None]
    if op == "shared":
        _, _, lens, _ = _shared_sizes(case)
        return _exact_attend(s, s["q"], lens, s["q_starts"].tolist())
    lens = _spread(case["seqs"], case["shortest"], case["longest"])
    q = _exact_rotate(s, s["q"], s["q_weight"])
    fresh = _exact_values(_exact_rotate(s, s["k"], s["k_weight"])), _exact_values(s["v"])
    # the attention takes the queries as they are handed over, in 16 bits
    return {"q": q, "out": _exact_attend(s, q.to(s["q"].dtype), lens, s["q_starts"].tolist(), fresh)}
