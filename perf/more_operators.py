"""Measured cases of decoding over a bounded paged cache: ``kv_append`` with
norms of the queries' and keys' heads, ``paged_attention`` through a sliding
window with first tokens that stay visible, and the pages' own operators:
``kv_free`` (pages that no token needs any more), ``kv_reserve`` (pages for new
tokens, with copies of shared pages that these are to be written into),
``kv_fork`` (sequences that go on from others, sharing their pages) and
``kv_compact`` (pages in use moved to the front of the pool).

``run`` computes a case in plain torch operations, or with ``own`` set through
the package's entry points; ``exact`` gives the outputs that are computed from
the operators' definitions in 64 bits.

The cache: pages of ``page`` tokens; keys ``[pages, kv heads, page, dim]`` and
values ``[pages, kv heads, dim, page]`` as E4M3 codes, one power-of-two scale
byte (exponent + 127) per page and head for each of the two.  ``table`` names
each sequence's pages (-1: none), ``refs`` counts the entries that name a page;
a page without any is free.  The caches of all layers share both.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # a decode batch at far positions, one norm weight for all heads
        {"name": "norm_append_decode", "op": "append", "dtype": "bf16", "hq": 32, "hkv": 8, "dim": 128, "page": 64,
         "batch": 64, "new": 1, "ctx": 131071, "rot": 128, "interleaved": False, "per_head": False},
        # three prompts of a prefill, ragged, part of the head rotated in neighbouring pairs, a weight for each head
        {"name": "norm_append_prefill", "op": "append", "dtype": "f16", "hq": 42, "hkv": 6, "dim": 128, "page": 128,
         "batch": 3, "new": 4096, "ctx": 4111, "rot": 96, "interleaved": True, "per_head": True},
        # a decode batch far into long sequences, of which each token sees four first and 4096 last ones
        {"name": "sinks_decode_batch", "op": "attention", "dtype": "bf16", "hq": 32, "hkv": 8, "dim": 128, "page": 64,
         "batch": 64, "new": 1, "ctx": 100003, "window": 4096, "sinks": 4},
        # a chunk of a prompt behind a longer part of it, sinks that end inside a page
        {"name": "sinks_chunk_1024", "op": "attention", "dtype": "f16", "hq": 42, "hkv": 6, "dim": 128, "page": 64,
         "batch": 2, "new": 1024, "ctx": 16384, "window": 2048, "sinks": 100},
        # a decode step: one sequence in 64 starts a page
        {"name": "reserve_decode_step", "op": "reserve", "layers": 2, "hkv": 4, "dim": 128, "page": 64, "pages": 4096,
         "batch": 64, "new": 1, "ctx": 2047, "shared": 1},
        # eight prompts of eight samples each go on: every sample needs its own copy of the last page
        {"name": "reserve_after_fork", "op": "reserve", "layers": 16, "hkv": 8, "dim": 128, "page": 64, "pages": 512,
         "batch": 64, "new": 1, "ctx": 1500, "shared": 8},
        # four prompts become four samples each
        {"name": "fork_samples", "op": "fork", "kind": "samples", "batch": 4, "group": 4, "page": 64, "ctx": 4000},
        # a step of beam search over long sequences: rows choose their parents within groups of eight
        {"name": "fork_beams", "op": "fork", "kind": "beams", "batch": 128, "group": 8, "page": 64, "ctx": 131072},
        # a decode step of a few sequences with a window: hardly a page to free
        {"name": "free_behind_window", "op": "free", "batch": 16, "page": 64, "ctx": 30011, "keep": 4096, "sinks": 4,
         "ended": 0},
        # a large batch of long sequences, a quarter of which has ended
        {"name": "free_ended", "op": "free", "batch": 256, "page": 64, "ctx": 131072, "keep": 0, "sinks": 0, "ended": 64},
        # a small pool, nearly full
        {"name": "compact_small", "op": "compact", "layers": 2, "hkv": 2, "dim": 64, "page": 32, "pages": 500,
         "batch": 16, "filled": 90},
        # a pool of which half has been freed all over
        {"name": "compact_half", "op": "compact", "layers": 4, "hkv": 8, "dim": 128, "page": 64, "pages": 2048,
         "batch": 32, "filled": 50},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attention", "attention", "attention", "reserve", "fork", "free", "compact"])
    dim, page = rng.choice([64, 128, 128, 192, 256]), rng.choice([16, 32, 64, 64, 128, 256])
    if op in ("append", "attention"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        while True:
            hkv = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
            c = {"op": op, "dtype": dtype, "hq": hkv * rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12, 16]), "hkv": hkv,
                 "dim": dim, "page": page, "batch": _log_int(rng, 1, 64)}
            kind = rng.choice(["decode", "decode", "verify", "prefill"])
            c["new"] = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _log_int(rng, 9, 4096)
            c["ctx"] = c["new"] - 1 + _log_int(rng, 1, 131072)
            if c["hq"] > 48:
                continue
            if op == "append":
                c["rot"] = rng.choice([dim, dim, dim // 2, 0])
                c["interleaved"] = rng.random() < 0.5
                c["per_head"] = rng.random() < 0.5
                if work(c)["bytes"] <= 2.7e8:
                    return c
            else:
                c["window"] = _log_int(rng, 16, 8192)
                c["sinks"] = _log_int(rng, 1, 500)
                w = work(c)
                columns = min(c["ctx"], c["window"] + c["new"] + c["sinks"] + 3 * page)
                if (w["flops"] <= 5.9e10 and w["bytes"] <= 5.3e8 and c["batch"] * c["hq"] * c["new"] * columns <= 6e8
                        and c["batch"] * hkv * dim * columns <= 3e8):
                    return c
    while True:
        layers, hkv = rng.choice([1, 2, 3, 4, 8, 16, 40]), rng.choice([1, 2, 3, 4, 8])
        if op == "fork":
            group = rng.randint(1, 8)
            c = {"op": op, "kind": rng.choice(["samples", "beams"]), "group": group, "page": page}
            c["batch"] = _log_int(rng, 1, 16) * (group if c["kind"] == "beams" else 1)
            c["ctx"] = _log_int(rng, 1, 131072)
        elif op == "free":
            c = {"op": op, "batch": _log_int(rng, 1, 256), "page": page, "ctx": _log_int(rng, 1, 131072),
                 "keep": rng.choice([0, _log_int(rng, 1, 16384)]), "sinks": rng.choice([0, _log_int(rng, 1, 500)])}
            c["ended"] = rng.randint(0, c["batch"])
        elif op == "reserve":
            c = {"op": op, "layers": layers, "hkv": hkv, "dim": dim, "page": page, "pages": _log_int(rng, 16, 16384),
                 "batch": _log_int(rng, 1, 64), "new": rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 2000)]),
                 "shared": rng.choice([1, 1, 2, 3, 8])}
            c["ctx"] = c["new"] - 1 + _log_int(rng, 1, 16384)
            _, _, _, held, wanted = _reserve_plan(c)
            if held + wanted > c["pages"]:
                continue
        else:
            c = {"op": op, "layers": layers, "hkv": hkv, "dim": dim, "page": page, "pages": _log_int(rng, 16, 16384),
                 "batch": _log_int(rng, 1, 64), "filled": rng.randint(1, 99)}
        large = max((x for x in listed() if x["op"] == op), key=lambda x: work(x)["bytes"])
        pool = layers * hkv * dim * page * 2 * c.get("pages", 0)
        if work(c)["bytes"] <= work(large)["bytes"] and pool <= 1 << 30:
            return c


# ---------------------------------------------------------------------------
# what a case holds
# ---------------------------------------------------------------------------

def _rng(case):
    """The same numbers for every seed, so that the work is the case's."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence: ragged, the first one at the case's own
    sizes."""
    r = _rng(case)
    new, ctx = [case["new"]], [max(case["ctx"], case["new"])]
    for _ in range(case["batch"] - 1):
        n = case["new"] if case["new"] <= 8 else r.randint(max(1, case["new"] // 4), case["new"])
        new.append(n)
        ctx.append(max(n, r.randint(max(1, case["ctx"] // 4), case["ctx"])))
    return new, ctx


def _reserve_plan(case):
    """new, ctx, the pages that each sequence holds, how many there are together, and how many the call takes."""
    page, share = case["page"], case["shared"]
    new, ctx = _lengths(case)
    ctx = [ctx[i - i % share] - new[i - i % share] + new[i] for i in range(len(ctx))]     # the same tokens before the new ones
    held = [-(-(c - n) // page) for n, c in zip(new, ctx)]
    together = sum(h for i, h in enumerate(held) if i % share == 0)
    wanted = 0
    for i, (n, c) in enumerate(zip(new, ctx)):
        rows = min(share, len(ctx) - (i - i % share))
        wanted += -(-c // page) - held[i] + (1 if (c - n) % page and rows > 1 else 0)
    return new, ctx, held, together, wanted


def _moves(case):
    used = max(1, case["pages"] * case["filled"] // 100)
    return used, used * (case["pages"] - used) // case["pages"]


def _free_plan(case):
    """Length, pages held and pages kept of each sequence."""
    r, page = _rng(case), case["page"]
    out = []
    for i in range(case["batch"]):
        n = r.randint(max(1, case["ctx"] // 4), case["ctx"]) if i else case["ctx"]
        held = -(-n // page)
        ended = i < case["ended"]
        keep = [not ended and (case["keep"] <= 0 or (j + 1) * page > n - case["keep"] or j * page < case["sinks"])
                for j in range(held)]
        # without a window nothing was freed before; with one, all but what a step's token leaves behind
        was = [case["keep"] <= 0 or k or (j + 1) * page > n - 1 - case["keep"] or j * page < case["sinks"]
               for j, k in enumerate(keep)]
        out.append((0 if ended else n, was, keep))
    return out


def _fork_lengths(case):
    r = _rng(case)
    return [case["ctx"]] + [r.randint(max(1, case["ctx"] // 4), case["ctx"]) for _ in range(case["batch"] - 1)]


def work(case):
    op = case["op"]
    if op == "fork":
        width = -(-case["ctx"] // case["page"])
        rows = case["batch"] * (case["group"] if case["kind"] == "samples" else 1)
        cells = (case["batch"] + rows) * width
        return {"bytes": 4 * (cells + 2 * sum(-(-n // case["page"]) for n in _fork_lengths(case))), "flops": cells}
    if op == "free":
        plan = _free_plan(case)
        cells = case["batch"] * -(-case["ctx"] // case["page"])
        gone = sum(sum(w) - sum(k) for _, w, k in plan)
        return {"bytes": 4 * (cells + 3 * gone), "flops": cells}
    if op in ("reserve", "compact"):
        page_bytes = case["layers"] * case["hkv"] * (2 * case["dim"] * case["page"] + 2)
        if op == "compact":
            _, moved = _moves(case)
            return {"bytes": 2 * moved * page_bytes + 12 * case["pages"], "flops": case["pages"]}
        new, ctx, held, _, _ = _reserve_plan(case)
        share, n = case["shared"], len(ctx)
        copies = sum(1 for i in range(n) if (ctx[i] - new[i]) % case["page"] and min(share, n - (i - i % share)) > 1)
        return {"bytes": 2 * copies * page_bytes + 4 * case["pages"] + 16 * n, "flops": case["pages"]}
    size = SIZES[case["dtype"]]
    new, ctx = _lengths(case)
    hq, hkv, dim, page = case["hq"], case["hkv"], case["dim"], case["page"]
    tokens = sum(new)
    if op == "append":
        # q in and out; k and v in, and their codes out
        bytes_ = tokens * dim * (2 * hq * size + 2 * hkv * (size + 1))
        return {"bytes": bytes_, "flops": tokens * (hq + hkv) * (3 * case["rot"] + 4 * dim) + tokens * hkv * dim * 4}
    pairs = read = 0
    window, sinks = case["window"], case["sinks"]
    for n, c in zip(new, ctx):
        for p in range(c - n, c):
            behind = max(0, p + 1 - window)
            pairs += p + 1 - behind + min(sinks, behind)
        behind = max(0, c - n + 1 - window)
        read += c - behind + min(sinks, behind)
    return {"bytes": 2 * tokens * hq * dim * size + 2 * read * hkv * dim + 2 * (read // page + 1) * hkv,
            "flops": 4 * dim * hq * pairs}


def _cache(case, pages, g):
    """A pool of pages filled with quantized values: ordinary keys and values, channels and heads of differing size."""
    hkv, page, dim = case["hkv"], case["page"], case["dim"]
    out = []
    for shape, channel in (((pages, hkv, page, dim), (1, hkv, 1, dim)), ((pages, hkv, dim, page), (1, hkv, dim, 1))):
        x = torch.randn(shape, device=DEV, generator=g, dtype=torch.bfloat16)
        x *= torch.exp(0.4 * torch.randn(channel, device=DEV, generator=g)).to(x.dtype)
        if case["op"] == "append":        # pages that are louder than the new tokens, and pages that are not
            x *= torch.exp2(torch.randint(-2, 2, (pages, hkv, 1, 1), device=DEV, generator=g).float()).to(x.dtype)
        byte = _scale_byte(x.abs().amax((2, 3)).float())
        x *= torch.exp2(127.0 - byte.float())[:, :, None, None].to(x.dtype)
        out.append((x.to(torch.float8_e4m3fn).view(torch.uint8), byte))
    (k, ks), (v, vs) = out
    return {"k": k, "v": v, "k_scales": ks, "v_scales": vs}


def _pools(case, g):
    """The layers' caches of a case that moves pages, side by side: any codes but NaN's."""
    pool, page, dim = (case["layers"], case["pages"], case["hkv"]), case["page"], case["dim"]

    def codes(*shape):
        return torch.randint(0, 127, shape, device=DEV, generator=g, dtype=torch.uint8)

    return {"k": codes(*pool, page, dim), "v": codes(*pool, dim, page), "k_scales": codes(*pool), "v_scales": codes(*pool)}


def _bookkeeping(s, table, refs):
    """The table and the pages' counts as one buffer: a pass works on a copy, since it changes them."""
    s["rows"], s["width"] = table.shape
    s["plan"] = torch.cat((table.flatten(), refs)).int().to(DEV)
    s["now"] = torch.empty_like(s["plan"])
    return s


def _restored(s):
    s["now"].copy_(s["plan"])
    cells = s["rows"] * s["width"]
    return s["now"][:cells].view(s["rows"], s["width"]), s["now"][cells:]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    if case["op"] in ("append", "attention"):
        return _prepare_tokens(case, seed, g)
    s = {"case": case}
    page = case["page"]
    if case["op"] == "reserve":
        new, ctx, held, together, _ = _reserve_plan(case)
        s["caches"] = _pools(case, g)
        table = torch.full((len(ctx), -(-max(ctx) // page)), -1, dtype=torch.int32)
        order, at = torch.randperm(case["pages"], generator=host).int(), 0
        for i, h in enumerate(held):
            if i % case["shared"] == 0:
                ids = order[at:at + h]
                at += h
            table[i, :h] = ids
        s["tokens"] = sum(new)
        s["cu"] = None
        if case["new"] > 1:
            s["cu"] = torch.tensor([0] + [sum(new[:i + 1]) for i in range(len(new))], dtype=torch.int32, device=DEV)
        s["lens"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    elif case["op"] == "compact":
        used, moved = _moves(case)
        pages, batch = case["pages"], case["batch"]
        s["caches"] = _pools(case, g)
        ids = torch.cat((torch.randperm(used, generator=host)[:used - moved],
                         used + torch.randperm(pages - used, generator=host)[:moved]))
        ids = ids[torch.randperm(used, generator=host)].int()
        width = -(-used // batch) + 4
        table = torch.full((batch, width), -1, dtype=torch.int32)
        for i, part in enumerate(ids.tensor_split(batch)):
            table[i, :len(part)] = part
        if batch > 1 and used >= batch:       # the second sequence begins with the first one's pages
            n = min(4, len(ids.tensor_split(batch)[0]))
            table[1, width - n:] = table[0, :n]
    elif case["op"] == "free":
        plan = _free_plan(case)
        width = -(-case["ctx"] // page)
        was = torch.zeros(len(plan), width, dtype=torch.bool)
        for i, (_, w, _) in enumerate(plan):
            was[i, :len(w)] = torch.tensor(w)
        table = torch.full(was.shape, -1, dtype=torch.int32)
        count = int(was.sum())
        table[was] = torch.randperm(count + count // 8 + 1, generator=host)[:count].int()
        case = {**case, "pages": count + count // 8 + 1}
        s["lens"] = torch.tensor([n for n, _, _ in plan], dtype=torch.int32, device=DEV)
    else:
        lens = _fork_lengths(case)
        held = [-(-n // page) for n in lens]
        width, batch, group = -(-case["ctx"] // page), case["batch"], case["group"]
        case = {**case, "pages": sum(held) + sum(held) // 8 + 1}
        order, at = torch.randperm(case["pages"], generator=host).int(), 0
        table = torch.full((batch, width), -1, dtype=torch.int32)
        for i, h in enumerate(held):
            table[i, :h] = order[at:at + h]
            at += h
        if case["kind"] == "samples":
            parent = torch.arange(batch * group) // group
        else:
            # beams have the same pages but for their last ones
            for i in range(batch):
                first = i - i % group
                same = max(0, min(held[i], held[first]) - 2)
                table[i, :same] = table[first, :same]
            base = torch.arange(batch) // group * group
            parent = base + (torch.rand(batch, generator=host) * (batch - base).clamp_max(group)).long()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["parent"] = parent.int().to(DEV)
    refs = torch.bincount(table[table >= 0].long(), minlength=case["pages"])
    s = _bookkeeping(s, table, refs)
    if own and "caches" in s:
        import nvfp4_quantized_matmul_amd as nv
        s["handles"] = [nv.KVCache(**{n: x[i] for n, x in s["caches"].items()}) for i in range(case["layers"])]
    return s


def _prepare_tokens(case, seed, g):
    dtype = DTYPES[case["dtype"]]
    new, ctx = _lengths(case)
    page, tokens = case["page"], sum(new)
    width = -(-max(ctx) // page)
    table = torch.full((len(new), width), -1, dtype=torch.int32)
    # only the pages that the call reads or writes are there
    own_pages = []
    for n, c in zip(new, ctx):
        last = -(-c // page)
        if case["op"] == "append":
            own_pages.append(list(range((c - n) // page, last)))
        else:
            first = max(0, c - n + 1 - case["window"]) // page
            own_pages.append([i for i in range(last) if i >= first or i * page < case["sinks"]])
    pages = sum(len(x) for x in own_pages)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).int()
    at = 0
    for i, x in enumerate(own_pages):
        table[i, x] = order[at:at + len(x)]
        at += len(x)
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    s = {"case": case, "cache": _cache(case, pages, g), "table": table.to(DEV),
         "lens": torch.tensor(ctx, dtype=torch.int32, device=DEV), "max_new": max(new),
         "cu": torch.tensor([0] + [sum(new[:i + 1]) for i in range(len(new))], dtype=torch.int32, device=DEV)}
    # q, k and v are the parts of one projection's rows; channels of the projection differ in size
    qkv = torch.randn(tokens, (hq + 2 * hkv) * dim, device=DEV, generator=g)
    if case["op"] == "append":
        qkv *= torch.exp(0.5 * torch.randn((hq + 2 * hkv) * dim, device=DEV, generator=g))
        for name, heads in (("q_norm", hq), ("k_norm", hkv)):
            shape = (heads, dim) if case["per_head"] else (dim,)
            s[name] = 1.0 + 0.3 * torch.randn(shape, device=DEV, generator=g)
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV).float() / max(case["rot"], 1))
        s["inv_freq"] = s["inv_freq"] if case["rot"] else None
    q, k, v = qkv.to(dtype).split([hq * dim, hkv * dim, hkv * dim], dim=1)
    s["q"] = q.unflatten(1, (hq, dim))
    if case["op"] == "append":
        s["k"], s["v"] = k.unflatten(1, (hkv, dim)), v.unflatten(1, (hkv, dim))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _cache_outputs(c):
    return {"k": c["k"].view(torch.float8_e4m3fn), "v": c["v"].view(torch.float8_e4m3fn),
            "k_scales": c["k_scales"], "v_scales": c["v_scales"]}


def _own_append(s):
    import nvfp4_quantized_matmul_amd as nv
    q = nv.kv_append(s["k"], s["v"], nv.KVCache(**s["cache"]), s["table"], s["lens"], q=s["q"], cu_q=s["cu"], max_q=s["max_new"],
                     inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                     eps=EPS)
    return {"q": q, **_cache_outputs(s["cache"])}


def _own_attention(s):
    import nvfp4_quantized_matmul_amd as nv
    return nv.paged_attention(s["q"], nv.KVCache(**s["cache"]), s["table"], s["lens"], cu_q=s["cu"], max_q=s["max_new"],
                              window=s["case"]["window"], sinks=s["case"]["sinks"])


def _own_reserve(s):
    import nvfp4_quantized_matmul_amd as nv
    table, refs = _restored(s)
    missing = nv.kv_reserve(s["handles"], table, s["lens"], refs, cu_q=s["cu"], tokens=s["tokens"])
    return {"missing": missing, "table": table, "refs": refs, **_cache_outputs(s["caches"])}


def _own_fork(s):
    import nvfp4_quantized_matmul_amd as nv
    table, refs = _restored(s)
    table, lens = nv.kv_fork(table, s["lens"], refs, s["parent"])
    return {"table": table, "lens": lens, "refs": refs}


def _own_free(s):
    import nvfp4_quantized_matmul_amd as nv
    case = s["case"]
    table, refs = _restored(s)
    nv.kv_free(table, s["lens"], refs, case["page"], keep=case["keep"], sinks=case["sinks"])
    return {"table": table, "refs": refs}


def _own_compact(s):
    import nvfp4_quantized_matmul_amd as nv
    table, refs = _restored(s)
    used, where = nv.kv_compact(s["handles"], table, refs)
    return {"used": used, "where": where, "table": table, "refs": refs, **_cache_outputs(s["caches"])}


def _scale_byte(amax):
    """Exponent + 127 of the smallest power of two p with amax <= 448 p."""
    m, e = torch.frexp(amax)
    byte = (e - 9 + (m > 0.875).int() + 127).clamp(0, 254)
    return torch.where(amax > 0, byte, torch.zeros_like(byte)).to(torch.uint8)


def _token_places(s):
    """Sequence and position of every new token."""
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return seq, t - cu[seq] + lens[seq] - (cu[seq + 1] - cu[seq])


def _normed(x, weight):
    x = x.double()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.double()


def _rotate(x, angle, interleaved):
    r = 2 * angle.shape[1]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _plain_append(s):
    # in 64 bits: angles of far positions, and keys next to the border of a scale
    case, cache = s["case"], s["cache"]
    page = case["page"]
    cu, lens, table = s["cu"].long(), s["lens"].long(), s["table"].long()
    q, k = _normed(s["q"], s["q_norm"]), _normed(s["k"], s["k_norm"])
    if case["rot"]:
        _, pos = _token_places(s)
        angle = pos[:, None].double() * s["inv_freq"].double()
        q, k = _rotate(q, angle, case["interleaved"]), _rotate(k, angle, case["interleaved"])
    q, k = q.float().to(s["q"].dtype), k.float()
    v = s["v"].float()
    # the page slots that the new tokens may reach: [sequences, pages, tokens of a page]
    first = lens - (cu[1:] - cu[:-1])
    slots = (s["max_new"] + page - 1) // page + 1
    p_idx = first[:, None] // page + torch.arange(slots, device=DEV)
    at = p_idx[..., None] * page + torch.arange(page, device=DEV)
    is_new = (at >= first[:, None, None]) & (at < lens[:, None, None])
    is_old = (at < first[:, None, None]) & is_new.any(-1, keepdim=True)
    ids = torch.gather(table, 1, p_idx.clamp(0, table.shape[1] - 1))
    touched = is_new.any(-1) & (p_idx < table.shape[1]) & (ids >= 0)
    row = (cu[:-1, None, None] + at - first[:, None, None]).clamp(0, q.shape[0] - 1)
    pages = cache["k"].shape[0]
    owner = torch.full((pages + 1,), -1, device=DEV)
    owner[torch.where(touched, ids, pages).flatten()] = torch.arange(ids.numel(), device=DEV)
    owner = owner[:pages]
    mine = owner >= 0
    at_page = owner.clamp_min(0)
    for x, codes, scales, shape in ((k, "k", "k_scales", (0, 2, 1, 3)), (v, "v", "v_scales", (0, 2, 3, 1))):
        x = x[row].flatten(0, 1).permute(shape)                       # slots laid out as the pages are
        grid = (1, 1, page, 1) if codes == "k" else (1, 1, 1, page)
        fresh = is_new.flatten(0, 1).view((-1,) + grid[1:])
        kept = is_old.flatten(0, 1).view((-1,) + grid[1:])
        x, fresh, kept = x[at_page], fresh[at_page], kept[at_page]
        new = _scale_byte(torch.where(fresh & x.isfinite(), x.abs(), 0.0).amax((2, 3)))
        old = cache[scales]
        byte = torch.maximum(new, torch.where(kept.any(-1).any(-1), old, torch.zeros_like(old)))
        up = torch.exp2(127.0 - byte.double())[:, :, None, None]
        was = cache[codes].view(torch.float8_e4m3fn).float()
        down = torch.exp2(old.double() - byte.double())[:, :, None, None]
        y = torch.where(fresh, (x.double() * up).float(), torch.where(kept, (was.double() * down).float(), was))
        y = y.to(torch.float8_e4m3fn).view(torch.uint8)
        cache[codes].copy_(torch.where(mine[:, None, None, None], y, cache[codes]))
        scales_new = torch.where(mine[:, None], byte, old)
        cache[scales].copy_(scales_new)
    return {"q": q, **_cache_outputs(cache)}


def _plain_attention(s):
    case, cache = s["case"], s["cache"]
    hkv, dim, page, window, sinks = case["hkv"], case["dim"], case["page"], case["window"], case["sinks"]
    group = case["hq"] // hkv
    q, cu, lens = s["q"], s["cu"].long(), s["lens"].long()
    batch, width = s["table"].shape
    most = s["max_new"]
    # rows of each sequence beside each other: [sequences, kv heads, tokens * group, dim]
    t = torch.arange(most, device=DEV)
    count = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + t).clamp(0, q.shape[0] - 1)
    rows = q.float()[row].view(batch, most, hkv, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, hkv, -1, dim)
    # the pages of the first tokens, and those from the one on that the first row's window begins in
    pos = lens[:, None] - count[:, None] + t
    front = min(-(-sinks // page), width)
    begin = ((lens - count + 1 - window).clamp_min(0) // page).clamp_min(front)
    slots = torch.cat((torch.arange(front, device=DEV).expand(batch, front),
                       begin[:, None] + torch.arange(min((window + most) // page + 2, width), device=DEV)), 1)
    ids = torch.gather(s["table"].long(), 1, slots.clamp_max(width - 1))
    there = (ids >= 0) & (slots < width)
    ids = ids.clamp_min(0)
    at = (slots[..., None] * page + torch.arange(page, device=DEV)).flatten(1)

    def values(codes, scales):
        x = cache[codes][ids].view(torch.float8_e4m3fn).float()
        return x * torch.exp2(cache[scales][ids].float() - 127)[..., None, None]

    k = values("k", "k_scales").permute(0, 2, 1, 3, 4).reshape(batch, hkv, -1, dim)
    see = (at[:, None] <= pos[..., None]) & there.repeat_interleave(page, 1)[:, None]
    see &= (at[:, None] > pos[..., None] - window) | (at[:, None] < sinks)
    see = see.repeat_interleave(group, 1)[:, None]
    score = torch.matmul(rows, k.transpose(2, 3)) * dim ** -0.5
    score = torch.where(see, score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top.isfinite(), top, 0.0))
    del score
    v = values("v", "v_scales").permute(0, 2, 1, 4, 3).reshape(batch, hkv, -1, dim)
    v = torch.where((at < lens[:, None])[:, None, :, None], v, 0.0)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    out = out.view(batch, hkv, most, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, most, hkv * group, dim)
    seq, at = _token_places(s)
    return out[seq, at - (lens - count)[seq]].to(q.dtype)


def _copy_pages(caches, src, dst):
    for x in caches.values():
        x.index_copy_(1, dst, x[:, src])


def _plain_reserve(s):
    table, refs = _restored(s)
    page, pages = s["case"]["page"], s["case"]["pages"]
    lens, (batch, width) = s["lens"].long(), table.shape
    new = (s["cu"][1:] - s["cu"][:-1]).long() if s["cu"] is not None else torch.ones_like(lens)
    first = lens - new
    slots = -(-s["case"]["new"] // page) + 1
    at = first[:, None] // page + torch.arange(slots, device=DEV)
    reached = (at * page < lens[:, None]) & (new[:, None] > 0) & (at < width)
    ids = torch.gather(table.long(), 1, at.clamp_max(width - 1))
    there = (ids >= 0) & (ids < pages)
    shared = there & (refs[ids.clamp(0, pages - 1)] > 1)
    need = reached & (~there | shared)
    count = need.sum(1)
    free = torch.nonzero(refs <= 0)[:, 0]
    served = (count.cumsum(0) <= free.numel()) | (count == 0)
    need &= served[:, None]
    b, i = torch.nonzero(need, as_tuple=True)
    fresh = free[:b.numel()]
    old = ids[b, i]
    was = shared[b, i]
    copied = was & (i == 0) & (first[b] % page != 0)
    table[b, at[b, i]] = fresh.int()
    refs[fresh] = 1
    refs.index_add_(0, old[was], torch.full_like(old[was], -1, dtype=torch.int32))
    _copy_pages(s["caches"], old[copied], fresh[copied])
    return {"missing": torch.where(served, 0, count).int(), "table": table, "refs": refs,
            **_cache_outputs(s["caches"])}


def _count(refs, ids, change):
    ids = ids.flatten().long()
    ids = torch.where((ids >= 0) & (ids < refs.numel()), ids, refs.numel())
    add = torch.zeros(refs.numel() + 1, dtype=torch.int32, device=DEV)
    add.index_add_(0, ids, torch.full_like(ids, change, dtype=torch.int32))
    refs += add[:-1]


def _plain_fork(s):
    table, refs = _restored(s)
    parent = s["parent"].long()
    known = (parent >= 0) & (parent < table.shape[0])
    parent = parent.clamp(0, table.shape[0] - 1)
    out = torch.where(known[:, None], table[parent], -1)
    lens = torch.where(known, s["lens"][parent], 0)
    _count(refs, out, 1)
    _count(refs, table, -1)
    return {"table": out, "lens": lens, "refs": refs}


def _plain_free(s):
    case = s["case"]
    table, refs = _restored(s)
    lens, page = s["lens"].long()[:, None], case["page"]
    begin = torch.arange(table.shape[1], device=DEV) * page
    keep = begin < lens
    if case["keep"] > 0:
        keep = keep & ((begin + page > lens - case["keep"]) | (begin < case["sinks"]))
    gone = ~keep & (table >= 0) & (table < refs.numel())
    _count(refs, torch.where(gone, table, -1), -1)
    table.copy_(torch.where(gone, -1, table))
    return {"table": table, "refs": refs}


def _plain_compact(s):
    table, refs = _restored(s)
    pages = refs.numel()
    inside = refs > 0
    used = inside.sum()
    page = torch.arange(pages, device=DEV)
    src = torch.nonzero(inside & (page >= used))[:, 0]
    dst = torch.nonzero(~inside & (page < used))[:, 0]
    where = torch.where(inside, page, -1)
    where[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    known = (table >= 0) & (table < pages)
    table.copy_(torch.where(known, where[table.clamp(0, pages - 1).long()], table))
    _copy_pages(s["caches"], src, dst)
    return {"used": used.int().view(1), "where": where.int(), "table": table, "refs": refs,
            **_cache_outputs(s["caches"])}


_PLAIN = {"append": _plain_append, "attention": _plain_attention, "reserve": _plain_reserve, "fork": _plain_fork,
          "free": _plain_free, "compact": _plain_compact}
_OWN = {"append": _own_append, "attention": _own_attention, "reserve": _own_reserve, "fork": _own_fork,
        "free": _own_free, "compact": _own_compact}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_table():
    t = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        t.append(float("nan") if c & 127 == 127 else -x if c & 128 else x)
    return torch.tensor(t, dtype=torch.float64, device=DEV)


def exact(case, seed):
    """Of the pages' operators nothing is computed: counts, places, and copies of codes."""
    if case["op"] == "append":
        return _exact_append(prepare(case, seed))
    if case["op"] == "attention":
        return _exact_attention(prepare(case, seed))
    return None


def _exact_append(s):
    case, cache, page = s["case"], s["cache"], s["case"]["page"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    e4m3 = _e4m3_table()
    half = case["rot"] // 2
    lane = torch.arange(half, device=DEV)
    ia, ib = (2 * lane, 2 * lane + 1) if case["interleaved"] else (lane, lane + half)
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    for x, w in ((q, s["q_norm"]), (k, s["k_norm"])):
        size = torch.linalg.vector_norm(x, dim=2, keepdim=True) ** 2 / case["dim"]
        x /= torch.sqrt(size + EPS)
        x *= w.double()
    codes = {n: e4m3[cache[n].int()] for n in ("k", "v")}
    bytes_ = {n: cache[n + "_scales"].int() for n in ("k", "v")}
    for b in range(len(lens)):
        lo, hi = cu[b], cu[b + 1]
        first = lens[b] - (hi - lo)
        if half:
            turn = torch.outer(torch.arange(first, lens[b], device=DEV, dtype=torch.float64), s["inv_freq"].double())
            c, n = torch.cos(turn)[:, None], torch.sin(turn)[:, None]
            for x in (q, k):
                a, d = x[lo:hi, :, ia], x[lo:hi, :, ib]
                x[lo:hi, :, ia], x[lo:hi, :, ib] = a * c - d * n, d * c + a * n
        for p in range(first // page, (lens[b] - 1) // page + 1):
            begin, end = max(first, p * page), min(lens[b], (p + 1) * page)
            rows = slice(lo + begin - first, lo + end - first)
            held, i = begin - p * page, table[b][p]
            for name, x in (("k", k[rows].transpose(0, 1)), ("v", v[rows].permute(1, 2, 0))):
                amax = x.abs().amax((1, 2)).float().double()
                byte = torch.ceil(torch.log2(amax / 448)).clamp(-127, 127).int() + 127
                page_codes = codes[name][i] if name == "k" else codes[name][i].transpose(1, 2)
                was = bytes_[name][i].clone()
                if held:
                    byte = torch.maximum(byte, was)
                    page_codes[:, :held] *= torch.exp2((was - byte).double())[:, None, None]
                y = x * torch.exp2(127.0 - byte.double())[:, None, None]
                page_codes[:, held:held + end - begin] = y if name == "k" else y.transpose(1, 2)
                bytes_[name][i] = byte
    return {"q": q, "k": codes["k"], "v": codes["v"], "k_scales": None, "v_scales": None}


def _exact_attention(s):
    case, cache, page = s["case"], s["cache"], s["case"]["page"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    e4m3 = _e4m3_table()
    q = s["q"].double()
    out = torch.zeros_like(q)
    group = case["hq"] // case["hkv"]
    for b in range(len(lens)):
        lo, hi, n = cu[b], cu[b + 1], lens[b]
        held = [i for i, p in enumerate(table[b][:-(-n // page)]) if p >= 0]
        ids = torch.tensor([table[b][i] for i in held], device=DEV)
        at = torch.cat([torch.arange(i * page, (i + 1) * page) for i in held]).to(DEV)
        pos = torch.arange(n - (hi - lo), n, device=DEV)[:, None]
        hidden = (at > pos) | ((at + case["window"] <= pos) & (at >= case["sinks"]))
        for h in range(case["hkv"]):
            k = e4m3[cache["k"][ids, h].int()] * torch.exp2(cache["k_scales"][ids, h].double() - 127)[:, None, None]
            v = e4m3[cache["v"][ids, h].int()] * torch.exp2(cache["v_scales"][ids, h].double() - 127)[:, None, None]
            k, v = k.reshape(-1, case["dim"]), v.transpose(1, 2).reshape(-1, case["dim"])
            for j in range(h * group, (h + 1) * group):
                z = (q[lo:hi, j] @ k.T / math.sqrt(case["dim"])).masked_fill_(hidden, float("-inf"))
                out[lo:hi, j] = torch.softmax(z, 1) @ v
    return out
