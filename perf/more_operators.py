"""A new token's way through an 8-bit cache, as measured cases: rotary positions, writing into a paged
cache of e4m3 codes with one power-of-two scale per block of tokens and head, reading rows of it back,
and the attention of new tokens (one a row, drafts, prompts, or with a list of tokens a query) over it.

`run` computes each in plain torch operations (32 bits, one rounding at the end) or, with `own` set,
through the library's entry points.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
LEAST_SCALE = -100  # exponent of a silent block's scale
LARGEST_BYTES = 1.7e9  # of keys and values in a drawn attention case
LARGEST_FLOPS = 6.5e12  # of a drawn attention case
SCORES = 1 << 29  # scores that the plain attention holds at a time


def listed():
    return [
        # Queries and keys of a decode batch, rotated in their fused projection's output.
        {"name": "rope_decode", "op": "rope", "n": 32, "heads": 72, "more": 8, "d": 128, "first": 0, "rot": 128,
         "pairs": "half", "scaled": False, "far": 32768, "x": "bf16", "out": "bf16"},
        # Indexer queries of the 8192-query prefill chunk into 8 bits: 64 of 128 dimensions, long-context frequencies.
        {"name": "rope_index_queries", "op": "rope", "n": 8192, "heads": 64, "more": 0, "d": 128, "first": 0, "rot": 64,
         "pairs": "interleaved", "scaled": True, "far": 131072, "x": "bf16", "out": "fp8"},
        # The chunk's indexer keys: one head.
        {"name": "rope_index_keys", "op": "rope", "n": 8192, "heads": 1, "more": 0, "d": 128, "first": 0, "rot": 64,
         "pairs": "interleaved", "scaled": True, "far": 131072, "x": "f32", "out": "fp8"},
        # The new tokens of a decode batch.
        {"name": "write_decode", "op": "write", "rows": 32, "n": 32, "L": 4096, "P": 64, "B": 64, "kv_heads": 8, "d": 128,
         "values": True},
        # A prefill chunk of 8192 tokens over three ragged sequences.
        {"name": "write_prefill", "op": "write", "rows": 3, "n": 8192, "L": 20000, "P": 128, "B": 32, "kv_heads": 8,
         "d": 128, "values": True},
        # The paged indexer keys of the 8 x 131072 workload into the indexer's own dense layout.
        {"name": "read_index_keys", "op": "read", "rows": 8, "n": 8 * 131072, "L": 131072, "P": 64, "B": 64, "kv_heads": 1,
         "d": 128, "values": False, "out": "fp8"},
        # A chat sequence's cache, brought back for a pass in bf16.
        {"name": "read_rows", "op": "read", "rows": 2, "n": 3999, "L": 2000, "P": 64, "B": 64, "kv_heads": 8, "d": 128,
         "values": True, "out": "bf16"},
        # One chat sequence on an idle server: the call's latency.
        {"name": "attend_one_row", "op": "attend", "rows": 1, "n": 1, "most": 1, "L": 2000, "P": 16, "B": 16, "kv_heads": 8,
         "heads": 32, "d": 128, "k": 0},
        # Long-context decode of the 8 x 131072 workload, dense layer, ragged lengths.
        {"name": "attend_long", "op": "attend", "rows": 8, "n": 8, "most": 1, "L": 131072, "P": 64, "B": 64, "kv_heads": 8,
         "heads": 64, "d": 128, "k": 0},
        # Five drafted tokens a sequence, to be verified in one step.
        {"name": "attend_drafts", "op": "attend", "rows": 16, "n": 80, "most": 5, "L": 32768, "P": 64, "B": 64, "kv_heads": 8,
         "heads": 64, "d": 128, "k": 0},
        # The last queries of a prompt of 32768 tokens, each with the 2048 tokens that the indexer selected for it.
        {"name": "attend_selected", "op": "attend", "rows": 1, "n": 512, "most": 512, "L": 32768, "P": 64, "B": 64,
         "kv_heads": 8, "heads": 64, "d": 128, "k": 2048},
        # A prefill chunk of 8192 tokens over three sequences with long histories.
        {"name": "attend_prompt", "op": "attend", "rows": 3, "n": 8192, "most": 2731, "L": 32768, "P": 128, "B": 32,
         "kv_heads": 8, "heads": 64, "d": 128, "k": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rope", "write", "read"])
    if op == "rope":
        d = rng.choice([64, 128, 128, 192])
        rot = rng.choice([d, d // 2, 64])
        heads = _log(rng, 1, 96)
        x, out = rng.choice([("bf16", "bf16"), ("bf16", "fp8"), ("f32", "fp8"), ("f32", "f32"), ("bf16", "f32")])
        return {"op": op, "n": _log(rng, 1, min(16384, 6e7 / (heads * d))), "heads": heads,
                "more": rng.choice([0, 0, 1, 8]), "d": d, "first": rng.choice([0, d - rot]), "rot": rot,
                "pairs": rng.choice(["half", "interleaved"]), "scaled": rng.random() < 0.5,
                "far": _log(rng, 32, 1 << 20), "x": x, "out": out}
    B = rng.choice([16, 32, 64, 128])
    P, d, kv = B * rng.choice([1, 1, 2, 3]), rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 5, 8])
    if op in ("write", "read"):
        n = _log(rng, 1, 20000)
        rows = _log(rng, 1, min(64, n))
        least = 2 * _up(n, rows) + 2  # the shortest row is half as long and holds its tokens
        L = _log(rng, least, max(least, min(40000, 2e8 / (rows * kv * d))))
        case = {"op": op, "rows": rows, "n": n, "L": L, "P": P, "B": B, "kv_heads": kv, "d": d,
                "values": rng.random() < 0.8}
        return case if op == "write" else {**case, "out": rng.choice(["bf16", "f32", "fp8"])}
    heads = kv * rng.choice([1, 2, 4, 7, 8, 12])
    kind = rng.choice(["one", "drafts", "prompt", "prompt", "listed"])
    L = _log(rng, 40, 131072)
    rows = _log(rng, 1, max(1, min(64, LARGEST_BYTES / (2 * L * kv * d))))
    most = {"one": 1, "drafts": rng.randint(2, 8), "prompt": 0, "listed": 0}[kind]
    k = _log(rng, 16, min(L, 8192)) if kind == "listed" else 0
    seen = k or L
    if not most:
        most = _log(rng, 1, max(1, min(L // 2, 4096, LARGEST_FLOPS / (4.0 * d * heads * rows * seen),
                                       1024 / rows if k else 1e9)))
    most = min(most, L // 2)
    n = rng.randint(max(rows, most), rows * most) if rows > 1 else most
    return {"op": op, "rows": rows, "n": n, "most": most, "L": L, "P": P, "B": B, "kv_heads": kv, "heads": heads, "d": d,
            "k": k}


def _up(a, b):
    return -(-a // b)


def _lengths(case):
    """Ragged lengths between L/2 and L, in the order of the rows."""
    L, rows = case["L"], case["rows"]
    return [L - i * (L // 2) // rows for i in range(rows)]


def _counts(case):
    """New (or read) tokens of each row: n over the rows as evenly as it goes, at most `most` and the row's length;
    with 16 rows and more the last one has none: padding of a captured batch."""
    rows, n = case["rows"], case["n"]
    got = _lengths(case)
    most = [min(x, case.get("most", x)) for x in got]
    if rows >= 16:
        most[-1] = 0
    counts, left = [0] * rows, n
    if case.get("most", 0) > 1:  # one row with the most of them
        counts[0] = min(most[0], left)
        left -= counts[0]
    for i in range(rows):
        share = _up(left, rows - i)
        more = min(most[i] - counts[i], share)
        counts[i] += more
        left -= more
    for i in range(rows):
        more = min(most[i] - counts[i], left)
        counts[i] += more
        left -= more
    return counts


_BYTES = {"bf16": 2, "f32": 4, "fp8": 1}


def work(case):
    op = case["op"]
    if op == "rope":
        cells = case["n"] * case["heads"]
        moved = cells * case["d"] * (_BYTES[case["x"]] + _BYTES[case["out"]]) + 4 * case["n"] * (1 + (case["out"] == "fp8"))
        return {"bytes": moved, "flops": cells * (3 * case["rot"] + (case["d"] if case["out"] == "fp8" else 0))}
    counts, kv, d = _counts(case), case["kv_heads"], case["d"]
    if op == "write":
        cells = sum(counts) * kv * d * (2 if case["values"] else 1)
        return {"bytes": 3 * cells, "flops": 2 * cells}
    if op == "read":
        cells = sum(counts) * kv * d * (2 if case["values"] else 1)
        scales = 4 * cells // d if case["out"] == "fp8" else 0
        return {"bytes": cells * (1 + _BYTES[case["out"]]) + scales, "flops": 0 if case["out"] == "fp8" else cells}
    heads, k = case["heads"], case["k"]
    seen = held = 0
    for c, n in zip(counts, _lengths(case)):
        each = [min(k, p + 1) if k else p + 1 for p in range(n - c, n)]
        seen += sum(each)
        held += min(n, sum(each)) if c else 0
    moved = held * kv * (2 * d + 8 / case["B"]) + 4 * held / case["P"]
    moved += sum(counts) * (heads * (4 * d + 4) + 4 * k)
    return {"bytes": int(moved), "flops": 4 * d * heads * seen}


# ------------------------------------------------------------------ inputs


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _codes(g, *shape):
    return (100 * _normal(g, *shape)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scales(g, *shape):
    return torch.exp2(torch.randint(-9, -5, shape, generator=g, device="cuda").float())


def _ints(values):
    return torch.tensor(values, device="cuda", dtype=torch.int32)


def _table(g, lengths, P, width, pages):
    """A page table of random distinct pages for rows of these lengths, -1 behind them."""
    need = _up(lengths, P)[:, None] > torch.arange(width, device="cuda")
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    return torch.where(need, ids[(need.flatten().cumsum(0) - 1).clamp(min=0).view_as(need)], -1)


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
BASE, FACTOR, ORIGINAL, FAST, SLOW = 10000.0, 40.0, 4096.0, 32.0, 1.0


def _frequencies(rot, scaled):
    """Radians a position of each pair; scaled: those that turn less than SLOW times in the original context are
    slowed down by FACTOR, those that turn more than FAST times stay, with a ramp between."""
    freq = [BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    if not scaled:
        return freq, 1.0
    at = [rot * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(BASE)) for turns in (FAST, SLOW)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot // 2 - 1)
    ramp = [min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0) for i in range(rot // 2)]
    return [f * (1 - r + r / FACTOR) for f, r in zip(freq, ramp)], 1 + 0.1 * math.log(FACTOR)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    if own:
        import long_context_pool_amd as misa

        s["misa"] = misa
    op = case["op"]
    if op == "rope":
        n, heads, d = case["n"], case["heads"], case["d"]
        loud = 1 + 7 * (torch.rand(d, generator=g, device="cuda") < 0.03)  # channels of outliers
        every = (_normal(g, n, heads + case["more"], d) * loud).to(_TYPES[case["x"]])
        s["x"] = every[:, :heads]
        s["pos"] = torch.randint(case["far"], (n,), generator=g, device="cuda").int()
        freq, s["amplitude"] = _frequencies(case["rot"], case["scaled"])
        if own:
            m = s["misa"]
            freq, s["amplitude"] = m.misa_rope_frequencies(m.rope_scaling(
                m.MISA_ROPE_PARTS if case["scaled"] else m.MISA_ROPE_PLAIN, case["rot"], BASE, FACTOR, ORIGINAL, FAST,
                SLOW))
            kinds = {"bf16": m.MISA_BF16, "f32": m.MISA_F32, "fp8": m.MISA_FP8_E4M3}
            s["spec"] = m.rope_spec(heads, d, case["first"], case["rot"],
                                    m.MISA_ROPE_HALF if case["pairs"] == "half" else m.MISA_ROPE_INTERLEAVED,
                                    kinds[case["x"]], kinds[case["out"]], (heads + case["more"]) * d, heads * d,
                                    s["amplitude"])
        s["freq"] = torch.tensor(freq, device="cuda", dtype=torch.float64)
        s["out"] = torch.empty(n, heads, d, device="cuda", dtype=_TYPES[case["out"]])
        s["scale"] = torch.empty(n, device="cuda") if case["out"] == "fp8" else None
        return s
    rows, kv, d, P, B = (case[x] for x in ("rows", "kv_heads", "d", "P", "B"))
    order = torch.randperm(rows, generator=g, device="cuda").tolist()
    lengths, counts = ([got[i] for i in order] for got in (_lengths(case), _counts(case)))
    s["tokens"] = list(zip(lengths, counts))  # a server's scheduler knows them
    s["lengths"] = _ints(lengths)
    s["offsets"] = _ints([sum(counts[:i]) for i in range(rows + 1)])
    width = _up(case["L"], P)
    pages = _up(sum(_up(x, P) for x in lengths) * 11, 10) + 1  # a tenth to spare
    s["table"] = _table(g, s["lengths"], P, width, pages)
    values = case.get("values", True)
    s["k"], s["k_scale"] = _codes(g, pages, kv, P, d), _scales(g, pages, kv, P // B)
    s["v"], s["v_scale"] = (_codes(g, pages, kv, P, d), _scales(g, pages, kv, P // B)) if values else (None, None)
    n = sum(counts)
    if op == "write":
        s["k_new"] = _normal(g, n, kv, d).bfloat16()
        s["v_new"] = (3 * _normal(g, n, kv, d)).bfloat16() if values else None
    elif op == "read":
        # the last tokens of each row; whole rows where that is all of them
        s["first"] = _ints([x - c for x, c in s["tokens"]])
        t = _TYPES[case["out"]]
        codes = case["out"] == "fp8"
        s["k_out"] = torch.empty(n, kv, d, device="cuda", dtype=t)
        s["v_out"] = torch.empty(n, kv, d, device="cuda", dtype=t) if values else None
        s["k_out_scale"] = torch.empty(n, kv, device="cuda") if codes else None
        s["v_out_scale"] = torch.empty(n, kv, device="cuda") if codes and values else None
    else:
        heads, k = case["heads"], case["k"]
        s["q"] = (2 * _normal(g, n, heads, d)).bfloat16()
        s["idx"] = None
        if k:  # k distinct tokens of each query's prefix, by position; -1 where it is shorter
            s["idx"] = torch.empty(n, k, device="cuda", dtype=torch.int32)
            i = 0
            for length, count in s["tokens"]:
                for a in range(0, count, 256):
                    last = length - count + torch.arange(a, min(a + 256, count), device="cuda")
                    key = torch.rand(last.numel(), length, generator=g, device="cuda")
                    key[torch.arange(length, device="cuda") > last[:, None]] = -1
                    top, at = key.topk(min(k, length), dim=1)
                    at = torch.where(top < 0, length, at).sort(dim=1).values
                    s["idx"][i:i + last.numel()] = -1
                    s["idx"][i:i + last.numel(), :at.shape[1]] = torch.where(at < length, at, -1).int()
                    i += last.numel()
        s["out"] = torch.empty(n, heads, d, device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.empty(n, heads, device="cuda")
    if own:
        m = s["misa"]
        s["cache"] = m.cache(rows, width, pages, P, kv, d, d, m.MISA_FP8_E4M3)
        if op == "attend":
            s["ws"] = torch.empty(m.misa_block_attend_workspace_bytes(s["cache"], B, heads, n, case["most"], k),
                                  device="cuda", dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ the operators


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_rope(s):
    s["misa"].misa_rope(s["spec"], s["case"]["n"], s["x"], s["pos"], s["freq"], s["out"], s["scale"])
    return s["out"], s["scale"]


def _own_write(s):
    s["misa"].misa_block_write(s["cache"], s["case"]["B"], s["k_new"].shape[0], s["offsets"], s["lengths"], s["k_new"],
                               s["v_new"], s["k"], s["k_scale"], s["v"], s["v_scale"], s["table"])
    return s["k"], s["k_scale"], s["v"], s["v_scale"]


def _own_read(s):
    m, out = s["misa"], s["case"]["out"]
    kind = m.MISA_BF16 if out == "bf16" else m.MISA_F32 if out == "f32" else m.MISA_FP8_E4M3
    m.misa_block_read(s["cache"], s["case"]["B"], s["k_out"].shape[0], kind, s["offsets"], s["first"], s["lengths"],
                      s["k"], s["k_scale"], s["v"], s["v_scale"], s["table"], s["k_out"], s["k_out_scale"], s["v_out"],
                      s["v_out_scale"])
    return s["k_out"], s["k_out_scale"], s["v_out"], s["v_out_scale"]


def _own_attend(s):
    c = s["case"]
    s["misa"].misa_block_attend(s["cache"], c["B"], c["heads"], s["q"].shape[0], c["most"], c["k"], c["d"] ** -0.5,
                                s["offsets"], s["q"], s["k"], s["k_scale"], s["v"], s["v_scale"], s["table"],
                                s["lengths"], s["idx"], s["out"], s["lse"], s["ws"])
    return s["out"], s["lse"]


def _plain_rope(s):
    c = s["case"]
    a, rot = c["first"], c["rot"]
    turn = s["pos"].double()[:, None] * s["freq"]  # 64 bits: far positions
    cos, sin = ((f(turn) * s["amplitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    y = s["x"].float().clone()
    part = y[..., a:a + rot]
    if c["pairs"] == "half":
        x0, x1 = part[..., :rot // 2], part[..., rot // 2:]
        part.copy_(torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1))
    else:
        x0, x1 = part[..., 0::2], part[..., 1::2]
        part.copy_(torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2))
    if c["out"] != "fp8":
        return y.to(_TYPES[c["out"]]), None
    top = y.abs().amax((1, 2))
    scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
    return (y / scale[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _places(s, first=None):
    """Row, position, page and slot of each new (or read) token."""
    P = s["case"]["P"]
    offsets, lengths = s["offsets"].long(), s["lengths"].long()
    i = torch.arange(sum(c for _, c in s["tokens"]), device="cuda")
    row = torch.searchsorted(offsets, i, right=True) - 1
    start = lengths - (offsets[1:] - offsets[:-1]) if first is None else first.long()
    pos = start[row] + i - offsets[row]
    return row, pos, s["table"][row, pos // P].long(), pos % P


def _least_scale(top):
    """The smallest power of two, 2^-100 at least, with top <= 448 * it."""
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.exp2(torch.where(top > 0, e, LEAST_SCALE).clamp(min=LEAST_SCALE).float())


def _plain_write(s):
    c = s["case"]
    P, B, kv = c["P"], c["B"], c["kv_heads"]
    row, pos, page, slot = _places(s)
    block = page * (P // B) + slot // B
    lengths, offsets = s["lengths"].long(), s["offsets"].long()
    start = lengths - (offsets[1:] - offsets[:-1])
    grown = torch.nonzero((start % B != 0) & (offsets[1:] > offsets[:-1])).flatten()  # rows that go on in a block
    begin = start[grown]
    old_page, old_block = s["table"][grown, begin // P].long(), begin % P // B
    for new, pool, scales in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
        if new is None:
            continue
        new, bits = new.float(), pool.view(torch.uint8)
        top = torch.zeros(scales.shape[0] * scales.shape[2], kv, device="cuda")
        top.scatter_reduce_(0, block[:, None].expand(-1, kv), new.abs().amax(-1), "amax")
        want = _least_scale(top)
        # tokens that the block already holds: their scale counts, and their codes are brought to the new one
        had = scales[old_page, :, old_block]  # [rows, kv]
        at = old_page * (P // B) + old_block
        want[at] = torch.maximum(want[at], had)
        slots = old_block[:, None] * B + torch.arange(B, device="cuda")  # [rows, B]
        here = (old_page[:, None, None], torch.arange(kv, device="cuda")[:, None], slots[:, None])
        codes = bits[here].view(pool.dtype)
        moved = (codes.float() * (had / want[at])[..., None, None]).to(pool.dtype)
        keep = (slots < (begin % P)[:, None])[:, None, :, None]
        bits[here] = torch.where(keep, moved.view(torch.uint8), codes.view(torch.uint8))
        unit = want[block]  # [tokens, kv]
        bits[page, :, slot] = (new / unit[..., None]).to(pool.dtype).view(torch.uint8)
        scales[page, :, slot // B] = unit
    return s["k"], s["k_scale"], s["v"], s["v_scale"]


def _plain_read(s):
    c = s["case"]
    _, _, page, slot = _places(s, s["first"])
    got = []
    for pool, scales in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        if pool is None:
            got += [None, None]
            continue
        codes = pool.view(torch.uint8)[page, :, slot].view(pool.dtype)
        unit = scales[page, :, slot // c["B"]]
        if c["out"] == "fp8":
            got += [codes, unit]
        else:
            got += [(codes.float() * unit[..., None]).to(_TYPES[c["out"]]), None]
    return got


def _cached(s, pool, scale, page, slot):
    """[kv, tokens, d] in 32 bits of the listed places."""
    head = torch.arange(s["case"]["kv_heads"], device="cuda")[:, None]
    x = s[pool].view(torch.uint8)[page, head, slot].view(torch.float8_e4m3fn).float()
    return x * s[scale][page, head, slot // s["case"]["B"]][..., None]


def _plain_attend(s):
    c = s["case"]
    P, kv, d, heads = c["P"], c["kv_heads"], c["d"], c["heads"]
    share = heads // kv
    n = s["q"].shape[0]
    out = torch.empty(n, heads, d, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(n, heads, device="cuda")
    i = 0
    for r, (length, count) in enumerate(s["tokens"]):
        if not count:
            continue
        every = torch.arange(length, device="cuda")
        step = 1 if c["k"] else max(1, SCORES // (heads * length))
        if not c["k"]:
            k = _cached(s, "k", "k_scale", s["table"][r].long()[every // P], every % P)
            v = _cached(s, "v", "v_scale", s["table"][r].long()[every // P], every % P)
            kt = k.transpose(1, 2).contiguous()
        for a in range(0, count, step):
            b = min(a + step, count)
            last = length - count + torch.arange(a, b, device="cuda")
            if c["k"]:
                at = s["idx"][i + a].long()
                seen = (at >= 0) & (at <= last)
                at = at.clamp(min=0)
                page = s["table"][r].long()[at // P]
                k, v = _cached(s, "k", "k_scale", page, at % P), _cached(s, "v", "v_scale", page, at % P)
                kt = k.transpose(1, 2).contiguous()
                seen = seen[None]
            else:
                seen = every <= last[:, None]
            q = s["q"][i + a:i + b].float().view(b - a, kv, share, d).transpose(0, 1).reshape(kv, -1, d)
            score = (torch.matmul(q, kt) * d ** -0.5).view(kv, b - a, share, -1)
            score = torch.where(seen[None, :, None], score, -math.inf)
            top = score.amax(-1, keepdim=True)
            p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(kv, (b - a) * share, -1), v).view(kv, b - a, share, d) / total
            out[i + a:i + b] = o.transpose(0, 1).reshape(b - a, heads, d).bfloat16()
            lse[i + a:i + b] = (top + torch.log(total)).squeeze(-1).transpose(0, 1).reshape(b - a, heads)
        i += count
    return out, lse


_plain = {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "attend": _plain_attend}
_own = {"rope": _own_rope, "write": _own_write, "read": _own_read, "attend": _own_attend}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "rope":
        x = s["x"].double()
        y = x.clone()
        for i in range(case["rot"] // 2):
            a = case["first"] + (i if case["pairs"] == "half" else 2 * i)
            b = a + (case["rot"] // 2 if case["pairs"] == "half" else 1)
            angle = s["pos"].double() * s["freq"][i]
            cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            y[..., a] = s["amplitude"] * (cos * x[..., a] - sin * x[..., b])
            y[..., b] = s["amplitude"] * (sin * x[..., a] + cos * x[..., b])
        if case["out"] != "fp8":
            return y, None
        unit = y.abs().flatten(1).max(1).values / 448
        unit[unit == 0] = 1
        return y / unit[:, None, None], unit
    if op in ("write", "read"):
        P, B = case["P"], case["B"]
        rows, pages, slots = [], [], []
        table = s["table"].tolist()
        for r, (length, count) in enumerate(s["tokens"]):
            for p in range(length - count, length):
                rows.append(r)
                pages.append(table[r][p // P])
                slots.append(p % P)
        row, page, slot = (torch.tensor(x, device="cuda", dtype=torch.long) for x in (rows, pages, slots))
        out = []
        for j in ("k", "v"):
            pool, scale = s[j], s[j + "_scale"]
            if pool is None:
                out += [None, None]
                continue
            if op == "read":
                code = pool.view(torch.uint8)[page, :, slot].view(pool.dtype).double()
                unit = scale.double()[page, :, slot // B]
                out += [code, unit] if case["out"] == "fp8" else [code * unit[..., None], None]
                continue
            value, unit, new = pool.double(), scale.double(), s[j + "_new"].double()
            i = 0
            for r, (length, count) in enumerate(s["tokens"]):
                at = length - count
                while at < length:  # a block of this row at a time
                    page_, block = table[r][at // P], at % P // B
                    end = min(length, (at // B + 1) * B)
                    part = new[i:i + end - at]
                    top = part.abs().amax((0, 2))
                    want = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=LEAST_SCALE))
                    low = at % B
                    if low:
                        want = torch.maximum(want, unit[page_, :, block])
                        held = value[page_, :, block * B:block * B + low]
                        held.mul_((unit[page_, :, block] / want)[:, None, None])
                    unit[page_, :, block] = want
                    value[page_, :, at % P:at % P + end - at] = (part / want[None, :, None]).transpose(0, 1)
                    i += end - at
                    at = end
            out += [value, unit]
        return tuple(out)
    if work(case)["flops"] > 2e13:
        return None
    P, B, kv = case["P"], case["B"], case["kv_heads"]
    share = case["heads"] // kv
    n = s["q"].shape[0]
    out = torch.zeros(n, case["heads"], case["d"], device="cuda", dtype=torch.float64)
    lse = torch.full((n, case["heads"]), -math.inf, device="cuda", dtype=torch.float64)
    i = 0
    for r, (length, count) in enumerate(s["tokens"]):
        at = torch.arange(length, device="cuda")
        page, slot = s["table"][r].long()[at // P], at % P
        for h in range(kv) if count else ():
            def cached(pool, scale):
                code = pool.view(torch.uint8)[page, h, slot].view(pool.dtype).double()
                return code * scale[page, h, slot // B].double()[:, None]

            k, v = cached(s["k"], s["k_scale"]), cached(s["v"], s["v_scale"])
            mine = slice(h * share, (h + 1) * share)
            step = 1 if case["k"] else max(1, SCORES // (8 * share * length))
            for a in range(0, count, step):
                b = min(a + step, count)
                q = s["q"][i + a:i + b, mine].double()
                if case["k"]:
                    chosen = s["idx"][i + a].long()
                    chosen = chosen[(chosen >= 0) & (chosen <= length - count + a)]
                    score = q @ k[chosen].T / math.sqrt(case["d"])
                    values = v[chosen]
                else:
                    score = (q.reshape(-1, case["d"]) @ k.T / math.sqrt(case["d"])).view(b - a, share, -1)
                    late = at > length - count + torch.arange(a, b, device="cuda")[:, None]
                    score.masked_fill_(late[:, None], -math.inf)
                    values = v
                lse[i + a:i + b, mine] = torch.logsumexp(score, -1)
                out[i + a:i + b, mine] = torch.softmax(score, -1) @ values
        i += count
    return out, lse
