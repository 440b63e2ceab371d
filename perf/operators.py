"""The serving operators around the indexer, as measured cases: attention of one
new token over a paged cache (every token, or the tokens an index list picks),
writing tokens into pages, a beam step's page bookkeeping and copies, pool
compaction, and the root-mean-square norm with residual and 8-bit output.

`run` computes each in plain torch operations (32 bits, one rounding at the
end) or, with `own` set, through the library's entry points.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
LARGEST_BYTES = 1.7e9  # of keys and values in a drawn attention case


def listed():
    return [
        # One chat sequence on an idle server: the call's latency.
        {"name": "attend_one_row", "op": "attend", "rows": 1, "L": 2000, "P": 16, "kv_heads": 8,
         "heads": 32, "dk": 128, "dv": 128, "k": 0, "fp8": False},
        # Long-context decode of the 8 x 131072 workload, dense layer, fp8 cache, ragged lengths.
        {"name": "attend_long_fp8", "op": "attend", "rows": 8, "L": 131072, "P": 64, "kv_heads": 8,
         "heads": 64, "dk": 128, "dv": 128, "k": 0, "fp8": True},
        # The 32 x 32768 decode workload with its k = 2048 selected tokens, one row of padding.
        {"name": "attend_selected", "op": "attend", "rows": 32, "L": 32768, "P": 64, "kv_heads": 8,
         "heads": 64, "dk": 128, "dv": 128, "k": 2048, "fp8": False},
        # The same selection over a latent cache: one shared row per token, values are its head part.
        {"name": "attend_latent", "op": "attend", "rows": 32, "L": 32768, "P": 64, "kv_heads": 1,
         "heads": 128, "dk": 576, "dv": 512, "k": 2048, "fp8": False},
        # The new tokens of a decode batch.
        {"name": "write_decode", "op": "write", "n": 32, "rows": 32, "L": 4096, "P": 64,
         "kv_heads": 8, "dk": 128, "dv": 128, "fp8": False},
        # A prefill chunk of 8192 tokens over three sequences, quantised on the way in.
        {"name": "write_prefill_fp8", "op": "write", "n": 8192, "rows": 3, "L": 20000, "P": 64,
         "kv_heads": 8, "dk": 128, "dv": 128, "fp8": True},
        # The residual stream of a decode batch into an 8-bit projection.
        {"name": "norm_decode", "op": "norm", "rows": 32, "n": 4096, "groups": 1, "residual": True,
         "out": "fp8", "x": "bf16"},
        # Indexer queries of the 8192-query prefill chunk: 64 heads of 128, one scale per token.
        {"name": "norm_index_queries", "op": "norm", "rows": 8192, "n": 8192, "groups": 64,
         "residual": False, "out": "fp8", "x": "bf16"},
        # A beam step of a small search: 8 losers freed, 8 winners forked, each extended by a token.
        {"name": "beam_small", "op": "beam", "parents": 8, "L": 2000, "P": 16, "planes": 4,
         "kv_heads": 8, "d": 128},
        # The same with 128 sequences and larger pages.
        {"name": "beam_large", "op": "beam", "parents": 128, "L": 4096, "P": 32, "planes": 2,
         "kv_heads": 4, "d": 128},
        # A small pool, 60 percent of it live.
        {"name": "compact_small", "op": "compact", "pages": 1000, "live": 60, "rows": 8, "P": 16,
         "planes": 2, "kv_heads": 2, "d": 128},
        # A large pool before it is shrunk.
        {"name": "compact_large", "op": "compact", "pages": 20000, "live": 45, "rows": 64, "P": 32,
         "planes": 2, "kv_heads": 4, "d": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "norm", "beam", "compact"])
    if op == "attend":
        dk, dv = rng.choice([(64, 64), (128, 128), (128, 128), (256, 256), (576, 512)])
        latent = dk != dv
        kv = 1 if latent else rng.choice([1, 2, 4, 5, 8])
        heads = kv * (rng.choice([16, 20, 64, 128]) if latent else rng.choice([1, 2, 4, 7, 8, 12, 16]))
        k = rng.choice([0, _log(rng, 16, 8192)])
        L = max(k, _log(rng, 1, 131072))
        P = rng.choice([1, 8, 16, 24, 64, 128])
        fp8 = rng.random() < 0.4
        per_row = L * kv * (dk if latent else dk + dv) * (1 if fp8 else 2)
        rows = _log(rng, 1, max(1, min(64, LARGEST_BYTES / per_row)))
        return {"op": op, "rows": rows, "L": L, "P": P, "kv_heads": kv, "heads": heads, "dk": dk,
                "dv": dv, "k": k, "fp8": fp8}
    if op == "write":
        dk, dv = rng.choice([(64, 64), (128, 128), (256, 256), (576, 512)])
        n = _log(rng, 1, 8192)
        rows = _log(rng, 1, min(64, n))
        kv = 1 if dk != dv else rng.choice([1, 2, 5, 8])
        least = 2 * _up(n, rows) + 2  # the shortest row is half as long and holds its new tokens
        L = _log(rng, least, max(least, min(20000, 2e8 / (rows * kv * dk))))
        return {"op": op, "n": n, "rows": rows, "L": L, "P": rng.choice([1, 8, 16, 24, 64, 128]), "kv_heads": kv,
                "dk": dk, "dv": dv, "fp8": rng.random() < 0.6}
    if op == "norm":
        groups = rng.choice([1, 1, 1, 8, 32, 64])
        n = groups * (_log(rng, 17, 16384) if groups == 1 else rng.choice([64, 128, 112]))
        return {"op": op, "rows": _log(rng, 1, min(16384, 6e7 / n)), "n": n, "groups": groups,
                "residual": rng.random() < 0.6, "out": rng.choice(["fp8", "fp8", "bf16"]),
                "x": rng.choice(["bf16", "bf16", "f32"])}
    if op == "beam":
        return {"op": op, "parents": _log(rng, 1, 128), "L": _log(rng, 30, 4096),
                "P": rng.choice([8, 16, 24, 32]), "planes": rng.choice([1, 2]),
                "kv_heads": rng.choice([1, 2, 4]), "d": rng.choice([64, 128])}
    return {"op": op, "pages": _log(rng, 50, 20000), "live": rng.randint(5, 95), "rows": _log(rng, 1, 64),
            "P": rng.choice([8, 16, 32]), "planes": rng.choice([1, 2]), "kv_heads": rng.choice([1, 3, 4]),
            "d": rng.choice([64, 128])}


def _up(a, b):
    return -(-a // b)


def _lengths(case, rows):
    """Ragged lengths between L/2 and L; a batch of 16 and more carries one empty row of padding."""
    got = [case["L"] - i * (case["L"] // 2) // rows for i in range(rows)]
    return got[:-1] + [0] if rows >= 16 and case["op"] == "attend" else got


def work(case):
    op = case["op"]
    if op == "attend":
        seen = sum(min(n, case["k"]) if case["k"] else n for n in _lengths(case, case["rows"]))
        per = case["dk"] if case["dk"] != case["dv"] else case["dk"] + case["dv"]
        b = 1 if case["fp8"] else 2
        scales = (4 if case["dk"] != case["dv"] else 8) * case["fp8"]
        heads, rows = case["heads"], case["rows"]
        moved = seen * case["kv_heads"] * (per * b + scales)
        moved += rows * heads * (2 * (case["dk"] + case["dv"]) + 4)
        moved += 4 * (seen if case["k"] else _up(seen, case["P"]))
        return {"bytes": moved, "flops": 2 * seen * heads * (case["dk"] + case["dv"])}
    if op == "write":
        n = case["n"] - case["n"] // 16
        per = case["kv_heads"] * (case["dk"] if case["dk"] != case["dv"] else case["dk"] + case["dv"])
        return {"bytes": n * per * (3 if case["fp8"] else 4), "flops": n * per * (4 if case["fp8"] else 0)}
    if op == "norm":
        e = 2 if case["x"] == "bf16" else 4
        o = 1 if case["out"] == "fp8" else 2
        cells = case["rows"] * case["n"]
        return {"bytes": cells * (e * (3 if case["residual"] else 1) + o), "flops": 6 * cells}
    page = 2 * case["planes"] * case["kv_heads"] * case["P"] * case["d"] * 2
    if op == "beam":
        got = _lengths(case, case["parents"])
        part = sum(n % case["P"] != 0 for n in got) / len(got)  # of the parents; winners are drawn from them
        pages = sum(_up(n, case["P"]) for n in got)
        return {"bytes": case["parents"] * part * 2 * page + 16 * pages, "flops": 0}
    live = case["pages"] * case["live"] // 100
    moves = live * (case["pages"] - live) / case["pages"]
    return {"bytes": moves * 2 * page + 4 * (3 * case["pages"] + 2.5 * live), "flops": 0}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _cells(g, fp8, *shape):
    """A pool of cached rows: bf16, or e4m3 codes."""
    if fp8:
        return (100 * _normal(g, *shape)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _scales(g, *shape):
    return (0.6 + 0.8 * torch.rand(shape, generator=g, device="cuda")) / 100


def _ints(values):
    return torch.tensor(values, device="cuda", dtype=torch.int32)


def _table(g, lengths, P, width, pages):
    """A page table of random distinct pages for rows of these lengths, -1 behind them."""
    need = _up(lengths, P)[:, None] > torch.arange(width, device="cuda")
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    return torch.where(need, ids[(need.flatten().cumsum(0) - 1).clamp(min=0).view_as(need)], -1)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op, P = case["op"], case.get("P")
    if op == "norm":
        rows, n = case["rows"], case["n"]
        dt = torch.bfloat16 if case["x"] == "bf16" else torch.float32
        loud = 1 + 15 * (torch.rand(n, generator=g, device="cuda") < 0.01)  # channels of outliers
        s["x"] = (_normal(g, rows, n) * loud).to(dt)
        s["residual"] = (2 * _normal(g, rows, n) * loud).to(dt) if case["residual"] else None
        s["weight"] = 0.5 + torch.rand(n // case["groups"], generator=g, device="cuda")
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["out"] = torch.empty(rows, n, device="cuda", dtype=torch.float8_e4m3fn if case["out"] == "fp8" else torch.bfloat16)
        s["scale"] = torch.empty(rows, device="cuda") if case["out"] == "fp8" else None
        return s
    if op == "compact":
        pages, rows = case["pages"], case["rows"]
        live = pages * case["live"] // 100
        width = _up(_up(live * 5, 4), rows)
        ids = torch.randperm(pages, generator=g, device="cuda")[:live]
        more = ids[torch.randint(live, (rows * width,), generator=g, device="cuda")]  # pages shared by two rows
        at = torch.arange(rows * width, device="cuda")
        flat = torch.where(at < live, ids[at.clamp(max=live - 1)], torch.where(at < live * 5 // 4, more, -1))
        s["table"] = flat.view(rows, width).int()
        s["refs"] = torch.bincount(flat[flat >= 0], minlength=pages).int()
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["map"] = torch.empty(pages, device="cuda", dtype=torch.int32)
        s["live"] = torch.empty(1, device="cuda", dtype=torch.int32)
        s["src"], s["dst"] = (torch.empty(max(1, pages // 2), device="cuda", dtype=torch.int32) for _ in range(2))
        s["k"], s["v"] = _page_bits(g, case, pages), _page_bits(g, case, pages)
        if own:
            _cache(s, rows, width, pages, case["d"], case["d"])
            s["ws"] = torch.empty(s["misa"].misa_page_workspace_bytes(s["cache"]), device="cuda", dtype=torch.uint8)
        return s
    if op == "beam":
        n = case["parents"]
        lengths = _ints(_lengths(case, n))[torch.randperm(n, generator=g, device="cuda")]
        width = _up(case["L"], P) + 1
        pages = int(sum(_up(x, P) for x in _lengths(case, n)) * 1.1) + 3 * n
        s["lengths"] = torch.cat([lengths, torch.zeros_like(lengths)])
        s["table"] = _table(g, s["lengths"], P, width, pages)
        s["refs"] = torch.zeros(pages, device="cuda", dtype=torch.int32)
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        s["parent"] = torch.randint(n, (n,), generator=g, device="cuda").int()
        s["child"] = n + torch.randperm(n, generator=g, device="cuda").int()
        s["one"] = torch.ones(n, device="cuda", dtype=torch.int32)
        s["src"], s["dst"], s["ok"], s["ok_more"] = (torch.empty_like(s["one"]) for _ in range(4))
        s["k"], s["v"] = _page_bits(g, case, pages), _page_bits(g, case, pages)
        _plain_beam(s)  # the children hold the pages of a step before
        s["parent"] = torch.randint(n, (n,), generator=g, device="cuda").int()
        if own:
            s["src"], s["dst"] = s["src"].int(), s["dst"].int()  # the plain step left 64-bit ids
            _cache(s, 2 * n, width, pages, case["d"], case["d"])
        return s
    # attention and writes: a pool with a tenth of spare pages
    rows, kv, dk, dv, fp8 = (case[x] for x in ("rows", "kv_heads", "dk", "dv", "fp8"))
    latent = dk != dv
    lengths = _ints(_lengths(case, rows))[torch.randperm(rows, generator=g, device="cuda")]
    width = _up(case["L"], P)
    pages = _up(sum(_up(x, P) for x in _lengths(case, rows)) * 11, 10) + 1
    s["lengths"], s["table"] = lengths, _table(g, lengths, P, width, pages)
    s["k"] = _cells(g, fp8, pages, kv, P, dk)
    s["v"] = None if latent else _cells(g, fp8, pages, kv, P, dv)
    s["k_scale"] = _scales(g, pages, kv, P) if fp8 else None
    s["v_scale"] = _scales(g, pages, kv, P) if fp8 and not latent else None
    if op == "write":
        n = case["n"]
        i = torch.arange(n, device="cuda")
        row = i * rows // n
        last = torch.searchsorted(row, row, right=True)  # one past the last token of this token's row
        pos = (lengths[row] - (last - i)).clamp(min=0)
        s["row"] = torch.where(i < n - n // 16, row, -1).int()  # the rest is a captured batch's padding
        s["pos"] = pos.int()
        s["k_new"] = _normal(g, n, kv, dk).bfloat16()
        s["v_new"] = None if latent else (3 * _normal(g, n, kv, dv)).bfloat16()
    else:
        heads, k = case["heads"], case["k"]
        s["q"] = (2 * _normal(g, rows, heads, dk)).bfloat16()
        s["idx"] = None
        if k:  # k distinct tokens of each row's prefix, by position; -1 where it is shorter
            key = torch.rand(rows, case["L"], generator=g, device="cuda")
            key[torch.arange(case["L"], device="cuda") >= lengths[:, None]] = -1
            top, at = key.topk(k, dim=1)
            at = torch.where(top < 0, case["L"], at).sort(dim=1).values
            s["idx"] = torch.where(at < case["L"], at, -1).int()
        s["out"] = torch.empty(rows, heads, dv, device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.empty(rows, heads, device="cuda")
    if own:
        _cache(s, rows, width, pages, dk, dv)
        if op == "attend":
            s["ws"] = torch.empty(s["misa"].misa_attend_workspace_bytes(s["cache"], heads, k), device="cuda", dtype=torch.uint8)
    return s


def _page_bits(g, case, pages):
    shape = (case["planes"], pages, case["kv_heads"], case["P"], case["d"])
    return torch.randint(-32768, 32768, shape, generator=g, device="cuda", dtype=torch.int16)


def _cache(s, rows, width, pages, dk, dv):
    import long_context_pool_amd as misa

    case = s["case"]
    s["misa"] = misa
    s["cache"] = misa.cache(rows, width, pages, case["P"], case["kv_heads"], dk, dv,
                            misa.MISA_FP8_E4M3 if case.get("fp8") else misa.MISA_BF16)
    if "planes" in case:  # the copied buffers: every layer's keys and values
        page = case["kv_heads"] * case["P"] * dk * 2
        s["buffers"] = misa.page_buffers([(s["k"], case["planes"], page), (s["v"], case["planes"], page)])


# ------------------------------------------------------------------ the operators


def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_attend(s):
    s["misa"].misa_attend(s["cache"], s["case"]["heads"], s["case"]["k"], s["case"]["dk"] ** -0.5, s["q"], s["k"],
                          s["k_scale"], s["v"], s["v_scale"], s["table"], s["lengths"], s["idx"], s["out"], s["lse"],
                          s["ws"])
    return s["out"], s["lse"]


def _own_write(s):
    s["misa"].misa_page_write(s["cache"], s["case"]["n"], s["row"], s["pos"], s["k_new"], s["v_new"], s["k"],
                              s["k_scale"], s["v"], s["v_scale"], s["table"])
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _own_norm(s):
    c = s["case"]
    m = s.get("misa")
    if m is None:
        import long_context_pool_amd as m

        s["misa"] = m
    m.misa_rms_norm(c["rows"], c["n"], c["groups"], m.MISA_BF16 if c["x"] == "bf16" else m.MISA_F32,
                    m.MISA_FP8_E4M3 if c["out"] == "fp8" else m.MISA_BF16, 1e-6, s["x"], s["residual"], s["weight"],
                    s["sum"], s["out"], s["scale"])
    return s["sum"], s["out"], s["scale"]


def _own_beam(s):
    m, c, n = s["misa"], s["cache"], s["case"]["parents"]
    m.misa_page_free(c, n, s["child"], s["table"], s["lengths"], s["refs"])
    m.misa_page_fork(c, n, s["parent"], s["child"], s["table"], s["lengths"], s["refs"], s["src"], s["dst"], s["ok"])
    m.misa_page_copy(s["buffers"], s["k"].shape[1], n, s["src"], s["dst"])
    m.misa_page_extend(c, n, s["child"], s["one"], s["table"], s["lengths"], s["refs"], s["ok_more"])
    return s["table"], s["lengths"], s["refs"], s["ok"], s["ok_more"], s["k"], s["v"]


def _own_compact(s):
    s["misa"].misa_page_compact(s["cache"], s["table"], s["refs"], s["table_out"], s["refs_out"], s["map"], s["live"],
                                s["src"], s["dst"], s["ws"])
    s["misa"].misa_page_copy(s["buffers"], s["case"]["pages"], s["case"]["pages"] // 2, s["src"], s["dst"])
    return s["table_out"], s["refs_out"], s["map"], s["live"], s["k"], s["v"]


def _plain_attend(s):
    c = s["case"]
    rows, kv, heads, P, dv = c["rows"], c["kv_heads"], c["heads"], c["P"], c["dv"]
    at = s["idx"].long() if c["k"] else torch.arange(s["table"].shape[1] * P, device="cuda").expand(rows, -1)
    page = s["table"].gather(1, at.clamp(min=0) // P).long()
    seen = (at >= 0) & (at < s["lengths"][:, None]) & (page >= 0)
    slot = at.clamp(min=0) % P
    page = page.clamp(min=0)

    def rows_of(pool, scale):  # [rows, kv, tokens, d]
        head = torch.arange(kv, device="cuda")[None, :, None]
        bits = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
        got = bits[page[:, None], head, slot[:, None]]
        got = got.view(pool.dtype).float()
        return got if scale is None else got * scale[page[:, None], head, slot[:, None]][..., None]

    k = rows_of(s["k"], s["k_scale"])
    v = k[..., :dv] if s["v"] is None else rows_of(s["v"], s["v_scale"])
    q = s["q"].float().view(rows, kv, heads // kv, c["dk"])
    score = torch.matmul(k, q.transpose(2, 3).contiguous()).transpose(2, 3) * c["dk"] ** -0.5
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, torch.where(seen[:, None, :, None], v, 0.0).contiguous()) / torch.where(total > 0, total, 1.0)
    return out.reshape(rows, heads, dv).bfloat16(), (top + torch.log(total)).reshape(rows, heads)


def _plain_write(s):
    P = s["case"]["P"]
    keep = s["row"] >= 0
    row, pos = s["row"][keep].long(), s["pos"][keep].long()
    page, slot = s["table"][row, pos // P].long(), pos % P
    for new, pool, scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
        if new is None:
            continue
        new = new[keep]
        if scale is None:
            pool[page, :, slot] = new
        else:
            code, unit = _e4m3(new.float())
            pool.view(torch.uint8)[page, :, slot] = code.view(torch.uint8)
            scale[page, :, slot] = unit
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _e4m3(x):
    """e4m3 codes and the scale of each row: its largest magnitude becomes 448."""
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
    return (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _plain_norm(s):
    c = s["case"]
    y = s["x"].float()
    total = None
    if c["residual"]:
        y = y + s["residual"].float()
        total = y.to(s["x"].dtype)
    parts = y.view(c["rows"], c["groups"], -1)
    z = parts * torch.rsqrt(parts.square().mean(-1, keepdim=True) + 1e-6) * s["weight"]
    z = z.view(c["rows"], c["n"])
    if c["out"] == "bf16":
        return total, z.bfloat16(), None
    code, scale = _e4m3(z)
    return total, code, scale


def _free_pages(refs, n):
    """How many pages are free, and the n lowest of them (any page behind those)."""
    free = refs <= 0
    ids = torch.argsort(free.int(), descending=True, stable=True)
    return free.sum(), ids[torch.arange(n, device="cuda").clamp(max=ids.numel() - 1)]


def _plain_beam(s):
    P, n = s["case"]["P"], s["case"]["parents"]
    table, lengths, refs = s["table"], s["lengths"], s["refs"]
    parent, child = s["parent"].long(), s["child"].long()
    at = torch.arange(table.shape[1], device="cuda")
    # free the children
    held = at < _up(lengths[child], P)[:, None]
    ids = table[child]
    refs.index_add_(0, ids.clamp(min=0).flatten(), -(held & (ids >= 0)).flatten().int())
    table[child] = torch.where(held, -1, ids)
    lengths[child] = 0
    # fork: whole pages are shared, a partly filled last page gets a copy of its own
    size, ids = lengths[parent], table[parent]
    whole, part = (size // P)[:, None], size % P != 0
    rank = part.cumsum(0)
    count, lowest = _free_pages(refs, n)
    ok = ~part | (rank <= count)
    new = lowest[(rank - 1).clamp(min=0)]
    last = (part & ok)[:, None] & (at == whole)
    shared = ok[:, None] & (at < whole)
    table[child] = torch.where(shared, ids, torch.where(last, new[:, None].int(), -1))
    refs.index_add_(0, ids.clamp(min=0).flatten(), (shared & (ids >= 0)).flatten().int())
    refs.index_add_(0, new, (part & ok).int())
    lengths[child] = torch.where(ok, size, 0)
    s["src"] = torch.where(part & ok, ids.gather(1, whole.clamp(max=table.shape[1] - 1).long())[:, 0], -1)
    s["dst"] = torch.where(part & ok, new, -1)
    _plain_copy(s)
    # one more token each
    size = lengths[child]
    more = size % P == 0
    rank = more.cumsum(0)
    count, lowest = _free_pages(refs, n)
    ok_more = (~more | (rank <= count)) & (size < at.numel() * P)
    new = lowest[(rank - 1).clamp(min=0)]
    table[child] = torch.where((more & ok_more)[:, None] & (at == (size // P)[:, None]), new[:, None].int(), table[child])
    refs.index_add_(0, new, (more & ok_more).int())
    lengths[child] = size + ok_more.int()
    return table, lengths, refs, ok.int(), ok_more.int(), s["k"], s["v"]


def _plain_copy(s):
    keep = s["src"] >= 0
    src, dst = s["src"][keep].long(), s["dst"][keep].long()
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]


def _plain_compact(s):
    refs, pages = s["refs"], s["case"]["pages"]
    live = refs > 0
    count = live.sum()
    at = torch.arange(pages, device="cuda")
    hole, mover = ~live & (at < count), live & (at >= count)
    holes = torch.argsort(hole.int(), descending=True, stable=True)  # ascending ids first
    movers = torch.argsort(mover.int(), descending=True, stable=True)
    half = max(1, pages // 2)
    valid = at[:half] < hole.sum()
    s["src"] = torch.where(valid, movers[:half], -1).int()
    s["dst"] = torch.where(valid, holes[:half], -1).int()
    to = holes[(mover.cumsum(0) - 1).clamp(min=0)]
    new = torch.where(live, torch.where(mover, to, at), -1)
    table = torch.where(s["table"] >= 0, new[s["table"].clamp(min=0).long()], -1).int()
    refs_out = torch.zeros_like(refs).index_add_(0, new.clamp(min=0), torch.where(live, refs, 0))
    _plain_copy(s)
    return table, refs_out, new.int(), count.int().view(1), s["k"], s["v"]


_plain = {"attend": _plain_attend, "write": _plain_write, "norm": _plain_norm, "beam": _plain_beam,
          "compact": _plain_compact}
_own = {"attend": _own_attend, "write": _own_write, "norm": _own_norm, "beam": _own_beam, "compact": _own_compact}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    op = case["op"]
    if op in ("beam", "compact"):
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "norm":
        y = s["x"].double() + (s["residual"].double() if case["residual"] else 0)
        total = y.clone() if case["residual"] else None
        size = case["n"] // case["groups"]
        weight = s["weight"].double()
        for i in range(case["groups"]):
            part = y[:, i * size:(i + 1) * size]
            part.mul_(weight / torch.sqrt((part ** 2).sum(1, keepdim=True) / size + 1e-6))
        if case["out"] == "bf16":
            return total, y, None
        unit = y.abs().max(1).values / 448
        unit[unit == 0] = 1
        return total, y / unit[:, None], unit
    if op == "write":
        # the rows that are written, before their rounding to 8 bits; every other row as it was
        out = [x if x is None else x.double() for x in (s["k"], s["v"], s["k_scale"], s["v_scale"])]
        row, pos, table = s["row"].tolist(), s["pos"].tolist(), s["table"].tolist()
        at = [(i, table[r][p // case["P"]], p % case["P"]) for i, (r, p) in enumerate(zip(row, pos)) if r >= 0]
        i, page, slot = (torch.tensor(x, device="cuda", dtype=torch.long) for x in zip(*at)) if at else [torch.empty(0, device="cuda", dtype=torch.long)] * 3
        for j, new in enumerate((s["k_new"], s["v_new"])):
            if new is None:
                continue
            new = new.double()[i]
            if out[j + 2] is not None:
                unit = new.abs().max(2).values / 448
                unit[unit == 0] = 1
                out[j + 2][page, :, slot] = unit
                new = new / unit[..., None]
            out[j][page, :, slot] = new
        return tuple(out)
    rows, kv, P = case["rows"], case["kv_heads"], case["P"]
    share = case["heads"] // kv
    out = torch.zeros(rows, case["heads"], case["dv"], device="cuda", dtype=torch.float64)
    lse = torch.full((rows, case["heads"]), -math.inf, device="cuda", dtype=torch.float64)
    for b in range(rows):
        n = int(s["lengths"][b])
        at = s["idx"][b].long() if case["k"] else torch.arange(n, device="cuda")
        at = at[(at >= 0) & (at < n)]
        if not at.numel():
            continue
        page, slot = s["table"][b].long()[at // P], at % P
        for h in range(kv):
            def cached(pool, scale):
                x = pool.view(torch.uint8)[page, h, slot].view(pool.dtype) if scale is not None else pool[page, h, slot]
                return x.double() if scale is None else x.double() * scale[page, h, slot].double()[:, None]

            k = cached(s["k"], s["k_scale"])
            v = k[:, :case["dv"]] if s["v"] is None else cached(s["v"], s["v_scale"])
            q = s["q"][b, h * share:(h + 1) * share].double()
            score = (q @ k.T) / math.sqrt(case["dk"])
            lse[b, h * share:(h + 1) * share] = torch.logsumexp(score, 1)
            out[b, h * share:(h + 1) * share] = torch.softmax(score, 1) @ v
    return out, lse
