"""Workloads of the MXFP4 operators: quantisation, product, paged KV cache, attention over it.

Each case runs in two forms on the same inputs.  With ``own`` false the
operators are written out in elementary float32 torch operations; with
``own`` true the same work goes through the package's public functions.
``exact`` evaluates the definitions in binary64 and is written apart from
both.

MXFP4: 32 consecutive elements of a row share an E8M0 scale 2^(E-127) with
E - 127 = floor(log2 max|x|) - 2, and each element is the nearest E2M1 value
(ties to even, saturating at 6) of x / scale.  Packed: byte j of a row holds
element 2j in its low nibble and 2j+1 in its high one.  Scales of a matrix
lie in tiles of 128 rows x 4 scale columns; those of the KV cache are
row-major next to its codes.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_FOUR = 17 / 32  # bytes of one element held in MXFP4: half a byte and 1/32 of a scale


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token's hidden state, as a decoding step quantises it
        {"name": "quantize token", "op": "quantize", "rows": 1, "cols": 5376, "dtype": "bf16"},
        # float32 matrix with an odd width (a calibration tensor)
        {"name": "quantize odd fp32", "op": "quantize", "rows": 1337, "cols": 2001, "dtype": "fp32"},
        # the MLP's activation for a few thousand tokens
        {"name": "quantize activation", "op": "quantize", "rows": 4096, "cols": 14336, "dtype": "bf16"},
        # the MLP's down projection for one token: the weight is the traffic
        {"name": "linear token", "op": "linear", "m": 1, "n": 5376, "k": 14336, "dtype": "bf16"},
        # the qkv projection for a batch of decoding sequences
        {"name": "linear batch", "op": "linear", "m": 61, "n": 21504, "k": 5376, "dtype": "fp16"},
        # the down projection over all tokens of a video: the largest case
        {"name": "linear video", "op": "linear", "m": 37810, "n": 5376, "k": 14336, "dtype": "bf16"},
        # a prompt of many short sequences goes into small pages and comes back
        {"name": "cache short", "op": "cache", "seqs": 64, "shortest": 1, "longest": 301, "kv_heads": 4, "dim": 64,
         "page": 16, "dtype": "fp16"},
        # a few long prompts
        {"name": "cache prompt", "op": "cache", "seqs": 3, "shortest": 2049, "longest": 16001, "kv_heads": 8,
         "dim": 128, "page": 64, "dtype": "bf16"},
        # one conversation decodes a token: latency
        {"name": "attend token", "op": "attend", "seqs": 1, "shortest": 1023, "longest": 1023, "queries": 1,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a batch of conversations of very different lengths decodes: the cache is the traffic
        {"name": "attend batch", "op": "attend", "seqs": 32, "shortest": 257, "longest": 32767, "queries": 1,
         "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # long conversations with a sliding window whose first tokens stay visible
        {"name": "attend window", "op": "attend", "seqs": 7, "shortest": 20011, "longest": 65537, "queries": 1,
         "q_heads": 16, "kv_heads": 16, "dim": 64, "page": 16, "window": 4096, "sinks": 4, "dtype": "fp16"},
        # two prompts are taken in by chunks behind what the cache already holds
        {"name": "attend chunk", "op": "attend", "seqs": 2, "shortest": 4099, "longest": 8192, "queries": 2048,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "cache", "attend", "attend"])
    if op == "quantize":
        cols = _log(rng, 33, 28672)
        rows = _log(rng, 1, max(1, min(37810, 58_000_000 // cols)))
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "linear":
        n, k = _log(rng, 65, 28672), _log(rng, 129, 14336)
        return {"op": op, "m": _log(rng, 1, 16384), "n": n, "k": k, "dtype": rng.choice(["bf16", "fp16"])}
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 7, 8])
    dim, page = rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "cache":
        longest = _log(rng, 16, 16384)
        seqs = _log(rng, 1, max(1, min(64, 40_000_000 // (longest * kv_heads * dim))))
        return {"op": op, "seqs": seqs, "shortest": _log(rng, 1, longest), "longest": longest, "kv_heads": kv_heads,
                "dim": dim, "page": page, "dtype": dtype}
    longest = _log(rng, 65, 32768)
    queries = 1 if rng.random() < 0.6 else _log(rng, 2, min(1024, longest))
    # the padded scores and the padded cache of the plain form bound the batch
    cost = max(longest * kv_heads * dim * 2, longest * kv_heads * group * queries)
    seqs = _log(rng, 1, max(1, min(32, 1_000_000_000 // cost)))
    window = 0 if rng.random() < 0.6 else _log(rng, 16, longest)
    return {"op": op, "seqs": seqs, "shortest": _log(rng, queries, longest), "longest": longest, "queries": queries,
            "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window,
            "sinks": rng.choice([0, 4, 37]) if window else 0, "dtype": dtype}


def _lens(case):
    """Lengths of the sequences, from longest to shortest in equal ratios."""
    n, lo, hi = case["seqs"], case["shortest"], case["longest"]
    return [hi] if n == 1 else [int(round(hi * (lo / hi) ** (b / (n - 1)))) for b in range(n)]


def _queries(case, lens):
    """New tokens of each sequence: all alike for one, else falling along the batch."""
    n = case["seqs"]
    return [min(lens[b], max(1, case["queries"] * (n - b) // n)) for b in range(n)]


def _visible(length, n, window, sinks):
    """(query, key) pairs that the mask leaves, and the keys that some query of the sequence sees."""
    lo = [0 if window == 0 else max(0, p - window + 1) for p in range(length - n, length)]
    pairs = sum(length - n + i + 1 - at + min(sinks, at) for i, at in enumerate(lo))
    return pairs, length - lo[0] + min(sinks, lo[0])


def work(case):
    op, s = case["op"], _BYTES[case["dtype"]]
    if op == "quantize":
        e = case["rows"] * case["cols"]
        return {"bytes": e * (2 * s + 2 * _FOUR), "flops": 0}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k * s + n * k * _FOUR + m * n * s, "flops": 2 * m * n * k}
    lens, d = _lens(case), case["dim"]
    if op == "cache":
        e = 2 * sum(lens) * case["kv_heads"] * d
        return {"bytes": e * (2 * s + 2 * _FOUR), "flops": 0}
    new = _queries(case, lens)
    seen = [_visible(length, n, case["window"], case["sinks"]) for length, n in zip(lens, new)]
    pairs, keys = sum(p for p, _ in seen), sum(k for _, k in seen)
    read = 2 * keys * case["kv_heads"] * d * _FOUR + sum(new) * d * (case["q_heads"] + 2 * case["kv_heads"]) * s
    return {"bytes": read + sum(new) * d * (case["q_heads"] * s + 2 * case["kv_heads"] * _FOUR),
            "flops": 4 * pairs * case["q_heads"] * d}


# ------------------------------------------- MXFP4 in elementary operations --

def _power(e):
    """2^(e - 127) in float32 for whole e in 0..254, from its bits."""
    e = e.to(torch.int32)
    return torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _encode(x):
    """float32 [..., 32 b] -> E2M1 codes (uint8, one an element) and E8M0 codes [..., b]."""
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = blocks.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    y = (blocks * _power(127 - e).unsqueeze(-1)).abs()
    code = torch.zeros_like(y, dtype=torch.uint8)
    code += y > 0.25
    code += y >= 0.75
    code += y > 1.25
    code += y >= 1.75
    code += y > 2.5
    code += y >= 3.5
    code += y > 5.0
    code += torch.signbit(blocks).to(torch.uint8) * 8
    return code.reshape(x.shape), (e + 127).to(torch.uint8)


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _decode(packed, scales):
    """Packed codes [..., d/2] and E8M0 codes [..., d/32] -> float32 [..., d]."""
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).to(torch.int32)
    two = code & 7  # 0 .5 1 1.5 2 3 4 6
    mag = torch.where(two < 4, two.float() * 0.5, torch.where(two < 6, two.float() - 2.0, two.float() * 2.0 - 8.0))
    val = torch.where(code >= 8, -mag, mag)
    return (val.reshape(*scales.shape, 32) * _power(scales).unsqueeze(-1)).flatten(-2)


def _round_trip(x):
    """The float32 values that MXFP4 holds for the rows of x."""
    cols = x.shape[-1]
    full = torch.nn.functional.pad(x.float(), (0, -cols % 32))
    code, e = _encode(full)
    return _decode(_pack(code), e)[..., :cols]


def _tile_offsets(rows, groups, device):
    """Byte of scale (r, c) in the 128-row x 4-column tiles, as [rows, 4 groups]."""
    r = torch.arange(rows, device=device).unsqueeze(1)
    c = torch.arange(4 * groups, device=device).unsqueeze(0)
    return ((r // 128) * groups + c // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4


# ------------------------------------------------------------------ inputs --

def _activation(shape, g):
    x = torch.randn(shape, generator=g, device="cuda")
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.001, x * 20, x)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "quantize":
        return {"case": case, "x": _activation((case["rows"], case["cols"]), g).to(dt)}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        rows, groups = -(-n // 128) * 128, -(-k // 128)
        w = torch.zeros(rows, groups * 128, device="cuda")
        w[:n, :k] = torch.randn((n, k), generator=g, device="cuda") * k ** -0.5
        code, e = _encode(w)
        e[n:] = 0
        scales = torch.empty(rows * groups * 4, dtype=torch.uint8, device="cuda")
        scales[_tile_offsets(rows, groups, "cuda")] = e
        return {"case": case, "x": _activation((m, k), g).to(dt), "w_codes": _pack(code), "w_scales": scales}
    # a cache whose pages are dealt in random order; whatever no sequence has
    # written (the rest of a last page, unused pages) holds arbitrary bytes
    lens, page, heads, d = _lens(case), case["page"], case["kv_heads"], case["dim"]
    counts = [-(-length // page) for length in lens]
    pages = sum(counts) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(counts), dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    new = lens if case["op"] == "cache" else _queries(case, lens)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).cuda()
    pos = torch.cat([torch.arange(length - n, length) for length, n in zip(lens, new)]).cuda()
    slots = table[seq, pos // page].long() * page + pos % page
    total = len(slots)
    chan = torch.ones(heads, d, device="cuda")
    chan[:, ::17] = 6.0  # keys have a few large channels
    state = {"case": case, "table": table, "slots": slots,
             "lens": torch.tensor(lens, dtype=torch.int32).cuda(),
             "starts": torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda(),
             "k": (torch.randn((total, heads, d), generator=g, device="cuda") * chan).to(dt),
             "v": torch.randn((total, heads, d), generator=g, device="cuda").to(dt)}
    for name, mul in (("k", chan), ("v", None)):
        shape = (pages, heads, page, d)
        if case["op"] == "cache":
            state[name + "_codes"] = torch.randint(0, 256, (*shape[:3], d // 2), generator=g, device="cuda",
                                                   dtype=torch.uint8)
            state[name + "_scales"] = torch.randint(0, 256, (*shape[:3], d // 32), generator=g, device="cuda",
                                                    dtype=torch.uint8)
            continue
        x = torch.randn(shape, generator=g, device="cuda")
        code, e = _encode(x if mul is None else x * mul.unsqueeze(1))
        state[name + "_codes"], state[name + "_scales"] = _pack(code), e
    if case["op"] == "attend":
        held = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
        for b, length in enumerate(lens):
            slot = torch.arange(length, device="cuda")
            held[table[b, slot // page].long(), slot % page] = True
        junk = torch.randint(0, 256, state["k_scales"].shape, generator=g, device="cuda", dtype=torch.uint8)
        for name in ("k_scales", "v_scales"):
            state[name] = torch.where(held[:, None, :, None], state[name], junk)
        state["q"] = torch.randn((total, case["q_heads"], d), generator=g, device="cuda").to(dt)
        state["q_starts"] = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        state["most"] = max(new)
    return state


# -------------------------------------------------------------- plain forms --

def _plain_linear(s):
    case = s["case"]
    n, k = case["n"], case["k"]
    rows, groups = -(-n // 128) * 128, -(-k // 128)
    e = s["w_scales"][_tile_offsets(rows, groups, "cuda")]
    w = _decode(s["w_codes"], e)[:n, :k]
    return (_round_trip(s["x"]) @ w.T).to(s["x"].dtype)


def _plain_write(s):
    page = s["case"]["page"]
    at, off = s["slots"] // page, s["slots"] % page
    (kc, ke), (vc, ve) = _encode(s["k"].float()), _encode(s["v"].float())
    s["k_codes"][at, :, off], s["k_scales"][at, :, off] = _pack(kc), ke
    s["v_codes"][at, :, off], s["v_scales"][at, :, off] = _pack(vc), ve


def _plain_gather(s, name):
    """The cache of every sequence, padded to the longest: float32 [seqs, heads, tokens, d], zeros past the end."""
    table = s["table"].long()
    x = _decode(s[name + "_codes"][table], s[name + "_scales"][table])  # [seqs, pages, heads, page, d]
    x = x.transpose(1, 2).flatten(2, 3)
    past = torch.arange(x.shape[2], device="cuda") >= s["lens"].unsqueeze(1)
    return x.masked_fill(past[:, None, :, None], 0.0)


def _plain_read(s):
    dt = s["k"].dtype
    held = torch.arange(s["table"].shape[1] * s["case"]["page"], device="cuda") < s["lens"].unsqueeze(1)
    return tuple(_plain_gather(s, name).transpose(1, 2)[held].to(dt) for name in ("k", "v"))


def _plain_attend(s):
    case = s["case"]
    group, d, window = case["q_heads"] // case["kv_heads"], case["dim"], case["window"]
    k, v = _plain_gather(s, "k"), _plain_gather(s, "v")
    seqs, heads, tokens, _ = k.shape
    new = s["q_starts"][1:] - s["q_starts"][:-1]
    i = torch.arange(s["most"], device="cuda")
    real = i < new.unsqueeze(1)  # [seqs, most]
    rows = (s["q_starts"][:-1].unsqueeze(1) + i).clamp(max=len(s["q"]) - 1).long()
    q = s["q"].float()[rows].reshape(seqs, -1, heads, group, d).permute(0, 2, 3, 1, 4)  # [seqs, heads, group, most, d]
    scores = (q.reshape(seqs, heads, -1, d) @ k.transpose(2, 3)).reshape(seqs, heads, group, -1, tokens) * d ** -0.5
    p = (s["lens"] - new).unsqueeze(1) + i
    j = torch.arange(tokens, device="cuda")
    seen = j <= p.unsqueeze(2)
    if window:
        seen = seen & ((j > p.unsqueeze(2) - window) | (j < case["sinks"]))
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    weight = (scores - top).exp()
    total = weight.sum(-1, keepdim=True)
    out = (weight.reshape(seqs, heads, -1, tokens) @ v).reshape(seqs, heads, group, -1, d)
    out = out / total.clamp(min=1e-37)
    return out.permute(0, 3, 1, 2, 4).reshape(seqs, -1, heads * group, d)[real].to(s["q"].dtype)


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "quantize":
            return _round_trip(state["x"]).to(state["x"].dtype)
        if op == "linear":
            return _plain_linear(state)
        _plain_write(state)
        return _plain_read(state) if op == "cache" else _plain_attend(state)
    import diffusion_transformer_mlp_gb300 as fc2
    if op == "quantize":
        return fc2.mxfp4_dequantize(fc2.mxfp4_quantize(state["x"]), state["x"].dtype)
    if op == "linear":
        w = fc2.MXFP4Tensor(state["w_codes"], state["w_scales"], case["n"], case["k"])
        return fc2.mxfp4_linear(state["x"], w)
    cache = fc2.MXFP4Cache(state["k_codes"], state["k_scales"], state["v_codes"], state["v_scales"])
    fc2.mxfp4_cache_write(cache, state["k"], state["v"], state["slots"])
    if op == "cache":
        return fc2.mxfp4_cache_read(cache, state["table"], state["starts"], len(state["slots"]), state["k"].dtype)
    return fc2.mxfp4_cache_attention(state["q"], cache, state["table"], state["lens"], q_starts=state["q_starts"],
                                     max_queries=state["most"], window=case["window"], sinks=case["sinks"])


# ----------------------------------------------------- definitions, binary64 --

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_power(e):
    """2^e in binary64 for whole e, from its bits (pow on the GPU is off by an ulp for some)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_round_trip(x):
    """MXFP4 of each row from its definition, in binary64: the quantum of the E2M1 grid at |y| is 1/2 below 2,
    1 below 4 and 2 above, and torch.round takes ties to even multiples of it, which are the even codes."""
    cols = x.shape[-1]
    b = torch.cat((x.double(), x.new_zeros(*x.shape[:-1], -cols % 32, dtype=torch.float64)), -1).unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -125)
    one = torch.floor(torch.log2(a))  # off by one where log2 rounds up to a whole number: put right below
    one = torch.where(_exact_power(one) > a, one - 1, torch.where(_exact_power(one + 1) <= a, one + 1, one))
    y = b.abs() / _exact_power(one - 2)
    quantum = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    y = (torch.round(y / quantum) * quantum).clamp(max=6.0)
    return (torch.copysign(y, b) * _exact_power(one - 2)).flatten(-2)[..., :cols]


def _exact_decode(packed, scales):
    """float64 values of packed codes [..., d/2] with E8M0 codes [..., d/32]."""
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), dtype=torch.float64, device=packed.device)
    lo, hi = grid[(packed % 16).long()], grid[(packed // 16).long()]
    x = torch.stack((lo, hi), -1).reshape(*packed.shape[:-1], -1)
    return x * _exact_power(scales.long() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    w = work(case)
    if w["flops"] > 2e12 or w["bytes"] > 1e9:
        return None
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_round_trip(s["x"])
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        rows, groups = -(-n // 128) * 128, -(-k // 128)
        tiles = s["w_scales"].reshape(rows // 128, groups, 32, 4, 4)  # panel, group, row % 32, row / 32, column
        e = tiles.permute(0, 3, 2, 1, 4).reshape(rows, groups * 4)
        return _exact_round_trip(s["x"]) @ _exact_decode(s["w_codes"], e)[:n, :k].T
    page, d = case["page"], case["dim"]
    new_k, new_v = _exact_round_trip(s["k"]), _exact_round_trip(s["v"])
    if case["op"] == "cache":
        return new_k, new_v
    lens, group = _lens(case), case["q_heads"] // case["kv_heads"]
    new, at, outs = _queries(case, lens), 0, []
    for b, (length, n) in enumerate(zip(lens, new)):
        pages = s["table"][b, :-(-length // page)].long()
        kv = []
        for codes, scales, fresh in (("k_codes", "k_scales", new_k), ("v_codes", "v_scales", new_v)):
            x = _exact_decode(s[codes][pages], s[scales][pages]).transpose(1, 2).flatten(0, 1)[:length].clone()
            x[length - n:] = fresh[at:at + n]
            kv.append(x)
        p = torch.arange(length - n, length, device="cuda").unsqueeze(1)
        j = torch.arange(length, device="cuda")
        hide = j > p
        if case["window"]:
            hide = hide | ((j <= p - case["window"]) & (j >= case["sinks"]))
        heads = []
        for h in range(case["q_heads"]):
            q = s["q"][at:at + n, h].double()
            scores = (q @ kv[0][:, h // group].T / math.sqrt(d)).masked_fill(hide, -math.inf)
            heads.append(torch.softmax(scores, -1) @ kv[1][:, h // group])
        outs.append(torch.stack(heads, 1))
        at += n
    return torch.cat(outs)
