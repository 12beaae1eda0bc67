"""Positions and the 4-bit cache of a serving step, as cases that can be measured.

Three operators, in the order in which one step of a decoder block uses them:

  rope      queries and keys turned by their positions, along one axis or several (time, height, width),
            and back (the gradient, or keys that move to another position)
  append    the same turn on the way into a paged cache, in bf16, MXFP8 or MXFP4, the values beside them
  paged     attention of a few new tokens of every sequence over an MXFP4 cache, with grouped heads and,
            where a case says so, a sliding window and first tokens that stay visible

With `own` false, `run` computes them in elementary torch operations, in 32 bits but for the angles, which
take 64; with `own` true it calls the package. `exact` has the same definitions once more, in 64 bits.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one stream and five draft rows far into a text: latency
        {"name": "rope-6", "op": "rope", "tokens": 6, "heads": 32, "heads_kv": 8, "dim": 128, "rot": 128,
         "pairs": "halves", "axes": 1, "mixed": False, "far": 1000003, "factor": 1.0, "inverse": False},
        # a picture's patches between its text, three axes taking turns, and a long context's factor
        {"name": "rope-1531-3axes", "op": "rope", "tokens": 1531, "heads": 28, "heads_kv": 4, "dim": 128, "rot": 128,
         "pairs": "halves", "axes": 3, "mixed": True, "far": 5003, "factor": 1.1386, "inverse": False},
        # the gradient of a picture tower's turn: narrow heads, height and width, neighbours as pairs
        {"name": "rope-16384-2axes-back", "op": "rope", "tokens": 16384, "heads": 16, "heads_kv": 16, "dim": 80,
         "rot": 80, "pairs": "neighbours", "axes": 2, "mixed": False, "far": 128, "factor": 1.0, "inverse": True},
        # eight streams of six verification rows into an 8-bit cache: latency
        {"name": "append-48-mxfp8", "op": "append", "tokens": 48, "heads": 64, "heads_kv": 8, "dim": 128, "rot": 128,
         "pairs": "halves", "axes": 1, "mixed": False, "far": 16411, "factor": 1.0, "page": 16, "fmt": "mxfp8"},
        # a middling prompt into a 4-bit cache, half of each head turned
        {"name": "append-3061-mxfp4", "op": "append", "tokens": 3061, "heads": 32, "heads_kv": 8, "dim": 128,
         "rot": 64, "pairs": "halves", "axes": 1, "mixed": False, "far": 70001, "factor": 1.0, "page": 32,
         "fmt": "mxfp4"},
        # a long prompt with pictures into a bf16 cache, out of the fused projection's rows
        {"name": "append-20011-3axes-bf16", "op": "append", "tokens": 20011, "heads": 32, "heads_kv": 8, "dim": 128,
         "rot": 128, "pairs": "halves", "axes": 3, "mixed": False, "far": 30011, "factor": 1.0, "page": 64,
         "fmt": "bf16"},
        # one stream's next token over a chat's length: latency
        {"name": "paged-1x1-4k", "op": "paged", "batch": 1, "rows": 1, "heads": 32, "heads_kv": 8, "dim": 128,
         "page": 16, "max_len": 4096, "window": 0, "sinks": 0},
        # eight streams with drafts, ragged lengths
        {"name": "paged-8x6-16k", "op": "paged", "batch": 8, "rows": 6, "heads": 64, "heads_kv": 8, "dim": 128,
         "page": 64, "max_len": 16411, "window": 0, "sinks": 0},
        # a large batch of a model with narrow heads whose layers see a window and four first tokens
        {"name": "paged-160x1-window", "op": "paged", "batch": 160, "rows": 1, "heads": 64, "heads_kv": 8, "dim": 64,
         "page": 16, "max_len": 5003, "window": 1024, "sinks": 4},
        # a middling batch with a few drafts each, 16 rows to a kv head
        {"name": "paged-31x4-8k", "op": "paged", "batch": 31, "rows": 4, "heads": 16, "heads_kv": 4, "dim": 128,
         "page": 32, "max_len": 8191, "window": 0, "sinks": 0},
        # few sequences with long contexts: the whole cost is reading the cache once
        {"name": "paged-4x1-128k", "op": "paged", "batch": 4, "rows": 1, "heads": 32, "heads_kv": 8, "dim": 128,
         "page": 32, "max_len": 131072, "window": 0, "sinks": 0},
        # a full batch at a chat's length
        {"name": "paged-256x1-4k", "op": "paged", "batch": 256, "rows": 1, "heads": 32, "heads_kv": 8, "dim": 128,
         "page": 64, "max_len": 4096, "window": 0, "sinks": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["rope", "append", "append", "paged", "paged", "paged"])
        heads_kv = rng.choice([1, 2, 4, 8])
        heads = heads_kv * rng.choice([1, 2, 4, 5, 7, 8])
        dim = rng.choice([64, 128])
        window = rng.choice([0, 0, _log_int(rng, 16, 8192) | 1])
        if op == "paged":
            case = {"op": op, "batch": _log_int(rng, 1, 256), "rows": rng.choice([1, 1, 2, 4, 6, 7]), "heads": heads,
                    "heads_kv": heads_kv, "dim": dim, "page": rng.choice([8, 16, 32, 64, 128]),
                    "max_len": _log_int(rng, 8, 131072) | 1, "window": window,
                    "sinks": rng.choice([0, 1, 4, _log_int(rng, 1, 300)]) if window else 0}
            if case["batch"] * case["max_len"] * heads_kv > 256 * 4096 * 8:
                continue
        else:
            if op == "rope":
                dim = rng.choice([64, 80, 96, 128, 256])
            case = {"op": op, "tokens": _log_int(rng, 1, 32768) | 1, "heads": heads, "heads_kv": heads_kv, "dim": dim,
                    "rot": rng.choice([dim, dim, dim // 2 // 16 * 16]), "pairs": rng.choice(["halves", "neighbours"]),
                    "axes": rng.choice([1, 1, 2, 3]), "mixed": rng.random() < 0.5, "far": _log_int(rng, 100, 2000000),
                    "factor": rng.choice([1.0, 1.0, 1.25])}
            if op == "rope":
                case["inverse"] = rng.random() < 0.4
            else:
                case["page"] = rng.choice([8, 16, 32, 64, 128])
                case["fmt"] = rng.choice(["bf16", "mxfp8", "mxfp4"])
        if _cost(case) <= most:
            return case


def _lengths(case):
    """The sequences' lengths of a case: whatever the seed, so that `work` can count them."""
    rng = random.Random("%s %s" % (case["batch"], case["max_len"]))
    return [case["max_len"]] + [rng.randint(max(1, case["max_len"] // 4), case["max_len"])
                                for _ in range(case["batch"] - 1)]


def _seen(q_pos, window, sinks):
    """How many keys the row at q_pos sees."""
    if q_pos < 0:
        return 0
    if not window:
        return q_pos + 1
    first = max(0, q_pos + 1 - window)
    return q_pos + 1 - first + min(sinks, first)


_WIDTH = {"bf16": 2, "mxfp8": 1 + 1 / 32, "mxfp4": 1 / 2 + 1 / 32}      # bytes of a stored value


def work(case):
    if case["op"] == "paged":
        keys = pairs = 0
        for n in _lengths(case):
            # one pass over what any of the rows sees
            first = max(0, n - case["rows"] + 1 - case["window"]) if case["window"] else 0
            keys += n - first + min(case["sinks"], first)
            pairs += sum(_seen(n - case["rows"] + r, case["window"], case["sinks"]) for r in range(case["rows"]))
        rows = case["batch"] * case["rows"] * case["heads"] * case["dim"]
        pages = sum(-(-n // case["page"]) for n in _lengths(case))
        return {"bytes": keys * 2 * case["heads_kv"] * case["dim"] * _WIDTH["mxfp4"] + 4 * rows + 4 * pages,
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    n, hkv = case["tokens"] * case["dim"], case["heads_kv"]
    turned = case["tokens"] * case["rot"] * (case["heads"] + hkv)
    if case["op"] == "rope":
        return {"bytes": 4 * n * (case["heads"] + hkv) + 4 * case["axes"] * case["tokens"], "flops": 3 * turned}
    # q in and out, k and v in, what is stored out
    return {"bytes": n * (4 * case["heads"] + 4 * hkv + 2 * hkv * _WIDTH[case["fmt"]]) + 4 * (1 + case["axes"]) * case["tokens"],
            "flops": 3 * turned + 2 * n * hkv}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


# The magnitudes of E2M1's codes 0 to 7, and halfway between neighbours: ties go to the even code.
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _scale_exponents(blocks, shift, most):
    """Per block the smallest s with max|x| <= qmax * 2^s, qmax = (1 + most / 2^23) * 2^shift."""
    bits = blocks.abs().amax(-1).view(torch.int32)
    exp = (bits >> 23) - 127 - shift + ((bits & 0x7FFFFF) > most).int()
    return torch.where(bits == 0, -127, exp.clamp(-127, 126))


def _quantise(x, fmt):
    """MX codes per 32 values of the last dimension, and the scales' bytes (2^(b - 127)). MXFP8: E4M3; MXFP4: E2M1, two
    to a byte, the even element's code in the low half."""
    blocks = x.float().unflatten(-1, (-1, 32))
    exp = _scale_exponents(blocks, 8, 0x600000) if fmt == "mxfp8" else _scale_exponents(blocks, 2, 0x400000)
    scaled = blocks * ((127 - exp) << 23).view(torch.float32).unsqueeze(-1)
    scales = (exp + 127).to(torch.uint8)
    if fmt == "mxfp8":
        return scaled.to(torch.float8_e4m3fn).flatten(-2), scales
    a = scaled.abs()
    code = (a > 0.25).to(torch.uint8)
    for at, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += a >= at if even else a > at
    code += torch.signbit(scaled).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _values4(codes, scales, table):
    """What MXFP4 codes stand for, in the table's type."""
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    scale = torch.exp2(scales.to(table.dtype) - 127)
    return (table[both.int()].unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)


def _code_values(st, codes):
    """E2M1 codes as the numbers they stand for, which E4M3 holds too: four codes at a time."""
    return st["four"][codes.view(torch.int16).int()].view(torch.float8_e4m3fn)


def _frequencies(case):
    """Every pair's frequency and axis. Axes in turns (mixed) or in sections; a section's frequencies are its own where
    there are two axes (a picture's), and go on where there are three."""
    half, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        axis = [0] * half
    elif case["mixed"]:
        axis = [i % axes for i in range(half)]
    else:
        axis = [min(axes - 1, i * axes // half) for i in range(half)]
    if axes == 2 and not case["mixed"]:
        own_place = [axis[:i].count(a) for i, a in enumerate(axis)]
        freq = [10000.0 ** (-j / axis.count(a)) for j, a in zip(own_place, axis)]
    else:
        freq = [500000.0 ** (-i / half) for i in range(half)]
    return freq, axis


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    hkv, dim = case["heads_kv"], case["dim"]
    channel = torch.exp(0.3 * _randn(g, dim))            # some channels are larger than others
    if case["op"] == "paged":
        batch, rows, heads, page = case["batch"], case["rows"], case["heads"], case["page"]
        lengths = _lengths(case)
        width = -(-case["max_len"] // page)
        used = [-(-n // page) for n in lengths]
        pages = sum(used) + 1
        order = torch.randperm(pages, generator=g, device="cuda").int()
        column = torch.arange(width, device="cuda")
        used_t = torch.tensor(used, device="cuda")
        begin = torch.cumsum(used_t, 0) - used_t
        place = (begin[:, None] + column).clamp(max=pages - 1)
        st["table"] = torch.where(column < used_t[:, None], order[place], -1).int().contiguous()
        st["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        st["q"] = (1.5 * _randn(g, batch, rows, heads, dim)).bfloat16()
        st["cache"] = []
        for _ in range(2):
            codes = torch.empty(pages, hkv, page, dim // 2, dtype=torch.uint8, device="cuda")
            scales = torch.empty(pages, hkv, page, dim // 32, dtype=torch.uint8, device="cuda")
            step = max(1, (1 << 27) // (hkv * page * dim))
            for a in range(0, pages, step):
                n = min(step, pages - a)
                codes[a:a + n], scales[a:a + n] = _quantise(_randn(g, n, hkv, page, dim).mul_(channel), "mxfp4")
            st["cache"] += [codes, scales]
        st["out"] = torch.empty_like(st["q"])
        st["e2m1"] = torch.tensor(_E2M1 + [-v for v in _E2M1], device="cuda")
    else:
        n, heads = case["tokens"], case["heads"]
        qkv = _randn(g, n, heads + 2 * hkv, dim).mul_(channel).bfloat16()       # the rows of a fused projection
        st["q"], st["k"], st["v"] = qkv[:, :heads], qkv[:, heads:heads + hkv], qkv[:, heads + hkv:]
        freq, axis = _frequencies(case)
        st["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        st["axis"] = torch.tensor(axis, device="cuda")
        # text that ends at `far`; with axes, a picture's rows and columns among it
        at = torch.arange(n, device="cuda") + max(0, case["far"] - n)
        wide = max(1, min(n, case["far"], 61))
        axes = [at, at // wide % 47 + (at[0] if case["axes"] == 3 else 0), at % wide + (at[0] if case["axes"] == 3 else 0)]
        st["pos"] = torch.stack(axes[-2:] if case["axes"] == 2 else axes[:case["axes"]]).int().contiguous()
        st["q_out"] = torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda")
        if case["op"] == "rope":
            st["k_out"] = torch.empty(n, hkv, dim, dtype=torch.bfloat16, device="cuda")
        else:
            page = case["page"]
            pages = -(-n // page) + 3
            st["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:n].sort().values.int()
            # dead rows: turned, but not stored
            st["slots"] = torch.where(torch.arange(n, device="cuda") % 16 == 11, -1, st["slots"])
            old = (pages, hkv, page, dim)
            st["cache"] = []
            for _ in range(2):
                values = _randn(g, *old).bfloat16()
                st["cache"] += [values] if case["fmt"] == "bf16" else list(_quantise(values, case["fmt"]))
            if case["fmt"] == "mxfp4":
                byte = torch.tensor(_E2M1 + [-v for v in _E2M1], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
                c = torch.arange(65536, device="cuda")
                st["four"] = torch.stack([byte[(c >> s) & 15] for s in (0, 4, 8, 12)], -1).contiguous().view(torch.int32).flatten()
    if own:
        from block_scaled_fp8_moe_gb300 import binding as B
        if "freq" in st:        # what a model builds once
            st["rotary"] = B.Rotary(freq, axis=axis, axes=case["axes"], interleaved=case["pairs"] == "neighbours",
                                    factor=case["factor"])
        if "cache" in st:       # the handle of the same tensors, which a user keeps beside them
            c = st["cache"]
            st["handle"] = B.KvCache(*c) if len(c) == 2 else B.KvCache(*(t.view(torch.uint8) for t in (c[0], c[2], c[1], c[3])))
    return st


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------
def _turn_of(st):
    """Cosines and sines [tokens, 1, rot / 2] of a case's positions: the angles in 64 bits."""
    angle = st["pos"][st["axis"]].double().t() * st["freq"]
    if st["case"].get("inverse"):
        angle = -angle
    factor = st["case"]["factor"]
    return [(f(angle) * factor).float().unsqueeze(1) for f in (torch.cos, torch.sin)]


def _turned(x, turn, case):
    cos, sin = turn
    rot = case["rot"]
    x = x.float()
    if case["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        parts = [a * cos - b * sin, a * sin + b * cos]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        parts = [torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)]
    return torch.cat(parts + [x[..., rot:]], -1)


def _plain_rope(st):
    turn = _turn_of(st)
    return {t: _turned(st[t], turn, st["case"]).bfloat16() for t in "qk"}


def _stored(st):
    """The cache as numbers: codes of 8 and 4 bits as the values they stand for."""
    c = st["cache"]
    if len(c) == 2:
        return {"k": c[0], "v": c[1]}
    e8 = torch.float8_e8m0fnu
    codes = c[::2] if st["case"]["fmt"] == "mxfp8" else [_code_values(st, t) for t in c[::2]]
    return {"k": codes[0], "k_scales": c[1].view(e8), "v": codes[1], "v_scales": c[3].view(e8)}


def _plain_append(st):
    case = st["case"]
    turn = _turn_of(st)
    keep = st["slots"] >= 0
    at = st["slots"][keep].long()
    page, fmt = case["page"], case["fmt"]
    new = [_turned(st["k"], turn, case)[keep], st["v"][keep]]
    new = [x.bfloat16() for x in new] if fmt == "bf16" else [t for x in new for t in _quantise(x, fmt)]
    for cache, rows in zip(st["cache"], new):
        flat = torch.uint8 if cache.element_size() == 1 else cache.dtype
        cache.view(flat)[at // page, :, at % page] = rows.view(flat)
    return {"q": _turned(st["q"], turn, case).bfloat16(), **_stored(st)}


def _plain_paged(st):
    case, c = st["case"], st["cache"]
    batch, rows, heads, dim = st["q"].shape
    hkv, window = case["heads_kv"], case["window"]
    table = st["table"].clamp(min=0).long()
    k, v = (_values4(a[table], b[table], st["e2m1"]).transpose(1, 2).reshape(batch, hkv, -1, dim)
            for a, b in ((c[0], c[1]), (c[2], c[3])))
    k_pos = torch.arange(k.shape[2], device="cuda")
    length = st["lengths"].view(-1, 1, 1)
    q_pos = length - rows + torch.arange(rows, device="cuda").view(1, -1, 1)
    see = (k_pos <= q_pos) & (q_pos >= 0)
    if window:
        see = see & ((q_pos - k_pos < window) | (k_pos < case["sinks"]))
    see = see.repeat_interleave(heads // hkv, 1).unsqueeze(1)
    v = v.masked_fill((k_pos >= length).unsqueeze(-1), 0)       # what lies behind a sequence's end is nobody's
    q = st["q"].float().view(batch, rows, hkv, -1, dim).transpose(1, 2).reshape(batch, hkv, -1, dim)
    s = (q @ k.transpose(-1, -2)).mul_(dim ** -0.5)
    s.masked_fill_(~see, -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = s.sum(-1, keepdim=True)
    o = (s @ v) / torch.where(total > 0, total, 1)              # rows that see nothing give zeros
    return o.view(batch, hkv, rows, -1, dim).transpose(1, 2).reshape(batch, rows, heads, dim).bfloat16()


def _own_rope(st):
    from block_scaled_fp8_moe_gb300 import binding as B
    q, k = B.moe_rope(st["rotary"], st["q"], st["k"], st["pos"], inverse=st["case"]["inverse"], q_out=st["q_out"],
                      k_out=st["k_out"])
    return {"q": q, "k": k}


def _own_append(st):
    from block_scaled_fp8_moe_gb300 import binding as B
    q = B.moe_rope_kv_append(st["rotary"], st["handle"], st["q"], st["k"], st["v"], st["pos"], st["slots"],
                             q_out=st["q_out"])
    return {"q": q, **_stored(st)}


def _own_paged(st):
    from block_scaled_fp8_moe_gb300 import binding as B
    c = st["case"]
    return B.moe_paged_attention(st["q"], st["handle"], st["table"], st["lengths"], c["max_len"], window=c["window"],
                                 sinks=c["sinks"], out=st["out"])


_PLAIN = {"rope": _plain_rope, "append": _plain_append, "paged": _plain_paged}
_OWN = {"rope": _own_rope, "append": _own_append, "paged": _own_paged}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _exact_turn(st, x, rows):
    """Rows of x as complex numbers times e^(i angle)."""
    case = st["case"]
    rot = case["rot"]
    x = x[rows].double()
    turned = x.clone()
    angle = torch.remainder(st["pos"][:, rows].double()[st["axis"]] * st["freq"][:, None], 2 * math.pi).t()[:, None]
    w = torch.polar(torch.full_like(angle, case["factor"]), -angle if case.get("inverse") else angle)
    if case["pairs"] == "halves":
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * w
        turned[..., :rot // 2], turned[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * w
        turned[..., :rot] = torch.view_as_real(z).flatten(-2)
    return turned


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] != "paged":
        bands = [slice(a, a + 2048) for a in range(0, case["tokens"], 2048)]
        q, k = (torch.cat([_exact_turn(st, st[t], b) for b in bands]) for t in "qk")
        if case["op"] == "rope":
            return {"q": q, "k": k}
        if case["fmt"] != "bf16":
            # codes and scales follow from decisions about whole blocks, not numbers that come near one
            return {"q": q, "k": None, "k_scales": None, "v": None, "v_scales": None}
        kept = (st["slots"] >= 0).nonzero().flatten()
        slots = st["slots"][kept].long()
        by_token = [t.double().transpose(1, 2).flatten(0, 1).index_copy(0, slots, x[kept].double())
                    for t, x in zip(st["cache"], (k, st["v"]))]
        k, v = (t.unflatten(0, (-1, case["page"])).transpose(1, 2) for t in by_token)
        return {"q": q, "k": k, "v": v}

    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    group, dim, page = case["heads"] // case["heads_kv"], case["dim"], case["page"]
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        pages = st["table"][b, :-(-n // page)].long()
        kv = []
        for codes, scales in (st["cache"][:2], st["cache"][2:]):
            codes = codes[pages].transpose(0, 1).flatten(1, 2)[:, :n].long()      # [heads_kv, n, dim / 2]
            values = torch.empty(*codes.shape[:2], dim, dtype=torch.float64, device="cuda")
            values[..., ::2], values[..., 1::2] = e2m1[codes % 16], e2m1[codes // 16]
            power = scales[pages].transpose(0, 1).flatten(1, 2)[:, :n].double() - 127
            kv.append(values * torch.pow(2.0, power).repeat_interleave(32, -1))
        keys = torch.arange(n, device="cuda")
        for r in range(case["rows"]):
            at = n - case["rows"] + r
            if at < 0:
                continue
            ok = keys <= at
            if case["window"]:
                ok &= (keys > at - case["window"]) | (keys < case["sinks"])
            q = st["q"][b, r].double().unflatten(0, (-1, group))
            s = torch.einsum("hgd,hnd->hgn", q, kv[0]) / math.sqrt(dim)
            s = torch.where(ok, s, torch.full_like(s, -math.inf))
            out[b, r] = torch.einsum("hgn,hnd->hgd", torch.softmax(s, -1), kv[1]).flatten(0, 1)
    return out
