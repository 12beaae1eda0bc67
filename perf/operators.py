"""The operators around the routed-expert layer in a serving step, as cases that can be measured.

Four operators, in the order in which one step of a decoder block uses them:

  append    the new tokens' keys and values into a paged cache, in bf16 or as MXFP8
  paged     attention of a few new tokens of every sequence over that cache, with grouped heads and,
            where a case says so, a sliding window and first tokens that stay visible
  prefill   attention of whole prompts, packed one behind the other, with the same window
  norm      the residual's addition, the root-mean-square norm and its MXFP8 quantisation, which is
            what the router and the experts' first product read

With `own` false, `run` computes them in elementary torch operations in 32 bits; with `own` true it
calls the package. `exact` has the same definitions once more, in 64 bits.
"""
import math
import random

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one stream and five draft rows between attention and the experts: latency
        {"name": "norm-6x4096", "op": "norm", "rows": 6, "cols": 4096, "residual": True},
        # a ragged batch of a narrower model, its first norm: nothing to add yet
        {"name": "norm-1531x2080", "op": "norm", "rows": 1531, "cols": 2080, "residual": False},
        # the largest prompt batch of the layer's own workloads
        {"name": "norm-32768x4096", "op": "norm", "rows": 32768, "cols": 4096, "residual": True},
        # eight streams of six verification rows into an 8-bit cache: latency
        {"name": "append-48-mxfp8", "op": "append", "tokens": 48, "heads_kv": 8, "dim": 128, "page": 16,
         "fmt": "mxfp8"},
        # a prompt's keys and values into a bf16 cache, out of the fused projection's rows
        {"name": "append-20011-bf16", "op": "append", "tokens": 20011, "heads_kv": 8, "dim": 128, "page": 64,
         "fmt": "bf16"},
        # one stream with its five drafts over a chat's length: latency
        {"name": "paged-1x6-4k-bf16", "op": "paged", "batch": 1, "rows": 6, "heads": 32, "heads_kv": 8, "dim": 128,
         "page": 16, "fmt": "bf16", "max_len": 4096, "window": 0, "sinks": 0},
        # eight streams with drafts, ragged lengths, 8-bit cache
        {"name": "paged-8x6-16k-mxfp8", "op": "paged", "batch": 8, "rows": 6, "heads": 64, "heads_kv": 8, "dim": 128,
         "page": 64, "fmt": "mxfp8", "max_len": 16411, "window": 0, "sinks": 0},
        # a large batch of a model with narrow heads whose layers see a window and four first tokens
        {"name": "paged-160x1-window-bf16", "op": "paged", "batch": 160, "rows": 1, "heads": 64, "heads_kv": 8,
         "dim": 64, "page": 16, "fmt": "bf16", "max_len": 5003, "window": 1024, "sinks": 4},
        # few sequences with long contexts: the whole cost is reading the cache once
        {"name": "paged-4x1-128k-bf16", "op": "paged", "batch": 4, "rows": 1, "heads": 32, "heads_kv": 8, "dim": 128,
         "page": 32, "fmt": "bf16", "max_len": 131072, "window": 0, "sinks": 0},
        # a handful of short prompts that came in together, down to single tokens
        {"name": "prefill-9x-1531-d64", "op": "prefill", "batch": 9, "tokens": 1531, "heads": 16, "heads_kv": 2,
         "dim": 64, "window": 128, "sinks": 4},
        # one prompt of the layer's 4k workload
        {"name": "prefill-1x-4096", "op": "prefill", "batch": 1, "tokens": 4096, "heads": 32, "heads_kv": 8,
         "dim": 128, "window": 1024, "sinks": 4},
        # long prompts of ragged lengths under a wide window
        {"name": "prefill-3x-12288", "op": "prefill", "batch": 3, "tokens": 12288, "heads": 32, "heads_kv": 8,
         "dim": 128, "window": 4096, "sinks": 64},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "append", "paged", "paged", "prefill", "prefill"])
        heads_kv = rng.choice([1, 2, 4, 8])
        heads = heads_kv * rng.choice([1, 2, 4, 5, 7, 8])
        dim = rng.choice([64, 128])
        window = rng.choice([0, _log_int(rng, 16, 8192) | 1])
        sinks = rng.choice([0, 1, 4, _log_int(rng, 1, 300)]) if window else 0
        if op == "norm":
            case = {"op": op, "rows": _log_int(rng, 1, 32768) | 1, "cols": 32 * (_log_int(rng, 2, 256) | 1),
                    "residual": rng.random() < 0.7}
        elif op == "append":
            case = {"op": op, "tokens": _log_int(rng, 1, 32768) | 1, "heads_kv": heads_kv, "dim": dim,
                    "page": rng.choice([8, 16, 32, 64, 128]), "fmt": rng.choice(["bf16", "mxfp8"])}
        elif op == "paged":
            case = {"op": op, "batch": _log_int(rng, 1, 192), "rows": rng.choice([1, 1, 2, 4, 6, 7]), "heads": heads,
                    "heads_kv": heads_kv, "dim": dim, "page": rng.choice([8, 16, 32, 64, 128]),
                    "fmt": rng.choice(["bf16", "mxfp8"]), "max_len": _log_int(rng, 8, 131072) | 1, "window": window,
                    "sinks": sinks}
            if case["batch"] * case["max_len"] * heads_kv > 4 * 131072 * 8:
                continue
        else:
            case = {"op": op, "batch": rng.choice([1, 2, 3, 5, 9]), "tokens": _log_int(rng, 16, 12288) | 1,
                    "heads": heads, "heads_kv": heads_kv, "dim": dim, "window": window, "sinks": sinks}
            # the plain form holds every score of every pair of rows
            if heads * case["tokens"] ** 2 > 32 * 12288 ** 2:
                continue
        if _cost(case) <= most:
            return case


def _lengths(case):
    """The sequences' lengths of a case: whatever the seed, so that `work` can count them."""
    rng = random.Random("%s %s %s" % (case["op"], case["batch"], case.get("max_len") or case.get("tokens")))
    n = case["batch"]
    if case["op"] == "paged":   # the longest has max_len tokens, the others less
        return [case["max_len"]] + [rng.randint(max(1, case["max_len"] // 4), case["max_len"]) for _ in range(n - 1)]
    cuts = sorted(rng.sample(range(1, case["tokens"]), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]


def _seen(q_pos, window, sinks):
    """How many keys the row at q_pos sees."""
    if q_pos < 0:
        return 0
    if not window:
        return q_pos + 1
    first = max(0, q_pos + 1 - window)
    return q_pos + 1 - first + min(sinks, first)


def _seen_sum(n, window, sinks):
    """The same, summed over the rows 0..n-1."""
    if not window or n <= window:
        return n * (n + 1) // 2
    behind = n - window                       # rows that no longer see their first keys
    low = min(behind, sinks)
    return window * (window + 1) // 2 + behind * window + low * (low + 1) // 2 + (behind - low) * sinks


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["cols"]
        # x (and the residual) in; the sum, the norm, its codes and its scales out
        return {"bytes": n * ((8 if case["residual"] else 6) + 1 + 1 / 32) + 2 * case["cols"], "flops": 8 * n}
    if op == "append":
        n = 2 * case["tokens"] * case["heads_kv"] * case["dim"]
        return {"bytes": n * (4 if case["fmt"] == "bf16" else 3 + 1 / 32) + 4 * case["tokens"], "flops": 2 * n}
    if op == "paged":
        per_key = 2 * case["heads_kv"] * case["dim"] * (2 if case["fmt"] == "bf16" else 1 + 1 / 32)
        keys = pairs = 0
        for n in _lengths(case):
            # one pass over what any of the rows sees
            if case["window"]:
                first = max(0, n - case["rows"] + 1 - case["window"])
                keys += n - first + min(case["sinks"], first)
            else:
                keys += n
            pairs += sum(_seen(n - case["rows"] + r, case["window"], case["sinks"]) for r in range(case["rows"]))
        rows = case["batch"] * case["rows"] * case["heads"] * case["dim"]
        pages = sum(-(-n // case["page"]) for n in _lengths(case))
        return {"bytes": keys * per_key + 4 * rows + 4 * pages, "flops": 4 * pairs * case["heads"] * case["dim"]}
    pairs = sum(_seen_sum(n, case["window"], case["sinks"]) for n in _lengths(case))
    rows = case["tokens"] * case["dim"]
    return {"bytes": 4 * rows * (case["heads"] + case["heads_kv"]), "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _mx_quantise(x):
    """MXFP8 per 32 values of the last dimension: the values as E4M3, the scales' bytes (2^(b - 127)).
    The scale is the smallest power of two with max|x| <= 448 * scale."""
    blocks = x.float().unflatten(-1, (-1, 32))
    bits = blocks.abs().amax(-1).view(torch.int32)
    exp = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    exp = torch.where(bits == 0, -127, exp.clamp(-127, 126))
    codes = (blocks * ((127 - exp) << 23).view(torch.float32).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes.flatten(-2), (exp + 127).to(torch.uint8)


def _mx_values(codes, scales, dtype):
    """What MXFP8 codes stand for."""
    scale = torch.exp2(scales.to(dtype) - 127)
    return (codes.to(dtype).unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        channel = torch.exp(0.5 * _randn(g, cols))               # some channels are much larger than others
        st["x"] = (_randn(g, rows, cols) * channel).bfloat16()
        st["residual"] = (3 * _randn(g, rows, cols) * channel).bfloat16() if case["residual"] else None
        st["weight"] = (1 + 0.1 * _randn(g, cols)).bfloat16()
        return st

    hkv, dim = case["heads_kv"], case["dim"]
    channel = torch.exp(0.3 * _randn(g, dim))
    if op == "append":
        n, page = case["tokens"], case["page"]
        pages = -(-n // page) + 3
        kv = _randn(g, n, 2 * hkv, dim).mul_(channel).bfloat16()    # the rows of a fused projection
        st["k"], st["v"] = kv[:, :hkv], kv[:, hkv:]
        st["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:n].sort().values.int()
        st["slots"] = torch.where(torch.arange(n, device="cuda") % 16 == 11, -1, st["slots"])  # dead rows: not stored
        old = (pages, hkv, page, dim)
        if case["fmt"] == "bf16":
            st["cache"] = [_randn(g, *old).bfloat16() for _ in range(2)]
        else:
            st["cache"] = [t for _ in range(2) for t in _mx_quantise(_randn(g, *old))]
    elif op == "paged":
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
            values = torch.empty(pages, hkv, page, dim, dtype=torch.bfloat16, device="cuda")
            values.normal_(generator=g).mul_(channel)
            st["cache"] += [values] if case["fmt"] == "bf16" else list(_mx_quantise(values))
        st["out"] = torch.empty_like(st["q"])
    else:
        n, heads = case["tokens"], case["heads"]
        st["q"] = _randn(g, n, heads, dim).mul_(channel).bfloat16()
        kv = _randn(g, n, 2 * hkv, dim).mul_(channel).bfloat16()    # the rows of a fused projection
        st["k"], st["v"] = kv[:, :hkv], kv[:, hkv:]
        lengths = _lengths(case)
        st["cu"] = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
        st["out"] = torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda")
    if own and "cache" in st:
        from block_scaled_fp8_moe_gb300 import binding as B
        c = st["cache"]         # the handle of the same tensors, which a user keeps beside them
        st["handle"] = B.KvCache(*c) if len(c) == 2 else B.KvCache(*(t.view(torch.uint8) for t in (c[0], c[2], c[1], c[3])))
    return st


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------
def _visible(q_pos, k_pos, window, sinks):
    see = k_pos <= q_pos
    if window:
        see = see & ((q_pos - k_pos < window) | (k_pos < sinks))
    return see & (q_pos >= 0)


def _attend(q, k, v, see):
    """q [..., rows, dim], k and v [..., keys, dim] in 32 bits; rows that see nothing give zeros."""
    s = (q @ k.transpose(-1, -2)).mul_(q.shape[-1] ** -0.5)
    s.masked_fill_(~see, -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = s.sum(-1, keepdim=True)
    return (s @ v) / torch.where(total > 0, total, 1)


def _plain_norm(st):
    h = st["x"].float() if st["residual"] is None else st["x"].float() + st["residual"].float()
    y = (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["weight"].float()).bfloat16()
    codes, scales = _mx_quantise(y)
    return {"sum": h.bfloat16(), "y": y, "codes": codes, "scales": scales.view(torch.float8_e8m0fnu)}


def _plain_append(st):
    keep = st["slots"] >= 0
    at = st["slots"][keep].long()
    page = st["case"]["page"]
    new = [st["k"][keep], st["v"][keep]]
    if st["case"]["fmt"] == "mxfp8":
        new = [t for x in new for t in _mx_quantise(x)]
    for cache, rows in zip(st["cache"], new):
        cache.view(torch.uint8 if cache.element_size() == 1 else cache.dtype)[at // page, :, at % page] = (
            rows.view(torch.uint8) if rows.element_size() == 1 else rows)
    return list(st["cache"])


def _plain_paged(st):
    case, c = st["case"], st["cache"]
    batch, rows, heads, dim = st["q"].shape
    hkv = case["heads_kv"]
    table = st["table"].clamp(min=0).long()
    if case["fmt"] == "bf16":
        k, v = c[0][table].float(), c[1][table].float()
    else:
        k, v = (_mx_values(a.view(torch.uint8)[table].view(torch.float8_e4m3fn), b[table], torch.float32)
                for a, b in ((c[0], c[1]), (c[2], c[3])))
    k, v = (t.transpose(1, 2).reshape(batch, hkv, -1, dim) for t in (k, v))
    k_pos = torch.arange(k.shape[2], device="cuda")
    length = st["lengths"].view(-1, 1, 1)
    q_pos = length - rows + torch.arange(rows, device="cuda").view(1, -1, 1)
    see = _visible(q_pos, k_pos, case["window"], case["sinks"]).repeat_interleave(heads // hkv, 1).unsqueeze(1)
    v = v.masked_fill((k_pos >= length).unsqueeze(-1), 0)       # what lies behind a sequence's end is nobody's
    q = st["q"].float().view(batch, rows, hkv, -1, dim).transpose(1, 2).reshape(batch, hkv, -1, dim)
    o = _attend(q, k, v, see)
    return o.view(batch, hkv, rows, -1, dim).transpose(1, 2).reshape(batch, rows, heads, dim).bfloat16()


def _plain_prefill(st):
    case = st["case"]
    n, heads, dim = st["q"].shape
    hkv = case["heads_kv"]
    row = torch.arange(n, dtype=torch.int32, device="cuda")
    seq = torch.bucketize(row, st["cu"][1:], right=True)
    see = (seq[:, None] == seq) & _visible(row[:, None], row, case["window"], 0)
    if case["window"]:
        pos = row - st["cu"][seq]
        see |= (seq[:, None] == seq) & (row <= row[:, None]) & (pos < case["sinks"])
    q = st["q"].float().view(n, hkv, -1, dim).permute(1, 2, 0, 3)
    k, v = (st[t].float().transpose(0, 1).unsqueeze(1) for t in "kv")
    return _attend(q, k, v, see).permute(2, 0, 1, 3).reshape(n, heads, dim).bfloat16()


def _own_norm(st):
    from block_scaled_fp8_moe_gb300 import binding as B
    y, total, codes, scales = B.moe_add_rmsnorm_mxfp8(st["x"], st["weight"], st["residual"], eps=EPS)
    return {"sum": total, "y": y, "codes": codes.view(torch.float8_e4m3fn),
            "scales": scales.view(torch.float8_e8m0fnu)}


def _own_append(st):
    from block_scaled_fp8_moe_gb300 import binding as B
    B.moe_kv_append(st["handle"], st["k"], st["v"], st["slots"])
    return list(st["cache"])


def _own_paged(st):
    from block_scaled_fp8_moe_gb300 import binding as B
    c = st["case"]
    return B.moe_paged_attention(st["q"], st["handle"], st["table"], st["lengths"], c["max_len"], window=c["window"],
                                 sinks=c["sinks"], out=st["out"])


def _own_prefill(st):
    from block_scaled_fp8_moe_gb300 import binding as B
    c = st["case"]
    return B.moe_prefill_attention(st["q"], st["k"], st["v"], st["cu"], window=c["window"], sinks=c["sinks"],
                                   out=st["out"])


_PLAIN = {"norm": _plain_norm, "append": _plain_append, "paged": _plain_paged, "prefill": _plain_prefill}
_OWN = {"norm": _own_norm, "append": _own_append, "paged": _own_paged, "prefill": _own_prefill}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _soft(q, k, v, see):
    """softmax(q k^T / sqrt(dim)) v of one head over the visible pairs, in 64 bits, in bands of rows."""
    out = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device="cuda")
    for a in range(0, q.shape[0], 2048):
        s = torch.einsum("id,jd->ij", q[a:a + 2048], k) / math.sqrt(q.shape[1])
        ok = see(a, min(a + 2048, q.shape[0]))
        s = torch.where(ok, s, torch.full_like(s, -math.inf))
        weight = torch.where(ok, torch.exp(s - torch.logsumexp(s, 1, keepdim=True)), torch.zeros_like(s))
        out[a:a + 2048] = weight @ v
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        parts = {"sum": [], "y": []}
        for a in range(0, case["rows"], 4096):
            h = st["x"][a:a + 4096].double()
            if case["residual"]:
                h = h + st["residual"][a:a + 4096].double()
            parts["sum"].append(h)
            parts["y"].append(h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["cols"] + EPS) * st["weight"].double())
        # codes and scales follow from the rounded norm: whole decisions, not numbers that come near one
        return {"sum": torch.cat(parts["sum"]), "y": torch.cat(parts["y"]), "codes": None, "scales": None}

    if op == "append":
        per = len(st["cache"]) // 2                              # codes and scales, or values alone
        outs = [t.double() if t.dtype != torch.uint8 else t for t in st["cache"]]
        kept = (st["slots"] >= 0).nonzero().flatten()
        slots = st["slots"][kept].long()
        for i, rows in enumerate((st["k"], st["v"])):
            new = [rows[kept].double()]
            if per == 2:
                # 448 * 2^power is the first such bound that no value of the block exceeds
                blocks = new[0].unflatten(-1, (-1, 32))
                power = torch.ceil(torch.log2(blocks.abs().amax(-1) / 448))
                new = [(blocks / torch.exp2(power).unsqueeze(-1)).flatten(-2), (power + 127).to(torch.uint8)]
            for j in range(per):
                by_token = outs[per * i + j].transpose(1, 2).flatten(0, 1).index_copy(0, slots, new[j])
                outs[per * i + j] = by_token.unflatten(0, (-1, case["page"])).transpose(1, 2)
        return outs

    window, sinks = case["window"], case["sinks"]

    def rule(first, count):
        keys = torch.arange(count, device="cuda")

        def see(a, b):
            q = torch.arange(first + a, first + b, device="cuda").unsqueeze(1)
            ok = (keys <= q) & (q >= 0)
            return ok & ((keys > q - window) | (keys < sinks)) if window else ok
        return see

    group = case["heads"] // case["heads_kv"]
    if op == "paged":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(case)):
            pages = st["table"][b, :-(-n // case["page"])].long()
            c = st["cache"]
            if case["fmt"] == "bf16":
                kv = [t[pages].double() for t in c]
            else:
                kv = [_mx_values(c[i].view(torch.uint8)[pages].view(torch.float8_e4m3fn), c[i + 1][pages],
                                 torch.float64) for i in (0, 2)]
            kv = [t.transpose(0, 1).flatten(1, 2)[:, :n] for t in kv]
            for r in range(case["rows"]):
                at = n - case["rows"] + r
                if at < 0:
                    continue
                for h in range(case["heads_kv"]):
                    ok = rule(at, n)(0, 1).expand(group, -1)
                    heads = slice(h * group, (h + 1) * group)
                    out[b, r, heads] = _soft(st["q"][b, r, heads].double(), kv[0][h], kv[1][h], lambda a, e: ok[a:e])
        return out

    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    begin = 0
    for n in _lengths(case):
        rows = slice(begin, begin + n)
        for h in range(case["heads"]):
            out[rows, h] = _soft(st["q"][rows, h].double(), st["k"][rows, h // group].double(),
                                 st["v"][rows, h // group].double(), rule(0, n))
        begin += n
    return out
