"""Measured cases of the serving operators around the quantized products:
``kv_append`` (rotation, 8-bit quantization and writing of new keys and values
into a paged cache), ``paged_attention`` (attention that reads that cache) and
``sample`` (the next token from its logits).

``run`` computes a case in plain torch operations, or with ``own`` set through
the package's entry points; ``exact`` gives the same outputs from the
operators' definitions in 64 bits.

The cache: pages of ``page`` tokens; keys ``[pages, kv heads, page, dim]`` and
values ``[pages, kv heads, dim, page]`` as E4M3 codes, one power-of-two scale
byte (exponent + 127) per page and head for each of the two.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one sequence decoding alone: a call of a few kilobytes, all latency
        {"name": "append_one_token", "op": "append", "dtype": "bf16", "hq": 32, "hkv": 8, "dim": 128, "page": 64,
         "batch": 1, "new": 1, "ctx": 1000, "rot": 128, "interleaved": False},
        # a decode batch at far positions, where 32-bit angles are off
        {"name": "append_decode_batch", "op": "append", "dtype": "bf16", "hq": 32, "hkv": 8, "dim": 128, "page": 64,
         "batch": 64, "new": 1, "ctx": 131071, "rot": 128, "interleaved": False},
        # three prompts of a prefill, ragged, part of the head rotated in neighbouring pairs
        {"name": "append_prefill", "op": "append", "dtype": "f16", "hq": 42, "hkv": 6, "dim": 128, "page": 128,
         "batch": 3, "new": 4096, "ctx": 4111, "rot": 96, "interleaved": True},
        # one sequence decoding alone over a short cache
        {"name": "decode_one_short", "op": "attention", "dtype": "bf16", "hq": 32, "hkv": 8, "dim": 128, "page": 64,
         "batch": 1, "new": 1, "ctx": 1003, "window": 0},
        # an ordinary decode batch, lengths ragged
        {"name": "decode_batch_8k", "op": "attention", "dtype": "bf16", "hq": 16, "hkv": 2, "dim": 128, "page": 64,
         "batch": 32, "new": 1, "ctx": 8191, "window": 0},
        # few sequences over very long caches: the long axis has to be split
        {"name": "decode_long_128k", "op": "attention", "dtype": "bf16", "hq": 32, "hkv": 8, "dim": 128, "page": 128,
         "batch": 4, "new": 1, "ctx": 131072, "window": 0},
        # speculative verification: a few tokens a sequence, float32, sliding window, wide heads
        {"name": "verify_window_f32", "op": "attention", "dtype": "f32", "hq": 21, "hkv": 7, "dim": 256, "page": 32,
         "batch": 16, "new": 6, "ctx": 4095, "window": 1024},
        # a whole prompt, causal
        {"name": "prefill_4096", "op": "attention", "dtype": "bf16", "hq": 42, "hkv": 6, "dim": 128, "page": 64,
         "batch": 1, "new": 4096, "ctx": 4096, "window": 0},
        # a chunk of a long prompt over what is cached of it, one head per kv head
        {"name": "chunk_1024_on_32k", "op": "attention", "dtype": "f16", "hq": 16, "hkv": 16, "dim": 64, "page": 256,
         "batch": 1, "new": 1024, "ctx": 32768, "window": 0},
        # one sequence's next token
        {"name": "sample_one_32k", "op": "sample", "dtype": "f32", "batch": 1, "vocab": 32000, "filters": "all"},
        # temperature and min-p alone, an odd vocabulary
        {"name": "sample_16_odd", "op": "sample", "dtype": "f16", "batch": 16, "vocab": 50001, "filters": "min_p"},
        # a decode batch over a large vocabulary, every row with its own settings
        {"name": "sample_64_256k", "op": "sample", "dtype": "bf16", "batch": 64, "vocab": 262144, "filters": "mixed"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    op = rng.choice(["append", "attention", "attention", "sample"])
    if op == "sample":
        return {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 64), "vocab": _log_int(rng, 1000, 262144),
                "filters": rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed"])}
    while True:
        hkv = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
        c = {"op": op, "dtype": dtype, "hq": hkv * rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12, 16]), "hkv": hkv,
             "dim": rng.choice([64, 128, 128, 256]), "page": rng.choice([32, 64, 64, 128, 256]),
             "batch": _log_int(rng, 1, 64)}
        kind = rng.choice(["decode", "decode", "verify", "prefill"])
        c["new"] = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _log_int(rng, 9, 4096)
        c["ctx"] = c["new"] - 1 + _log_int(rng, 1, 131072)
        if c["hq"] > 48:
            continue
        if op == "append":
            c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2])
            c["interleaved"] = rng.random() < 0.5
            if c["batch"] * c["new"] * (c["hq"] + 2 * hkv) * c["dim"] <= 1 << 26:
                return c
        else:
            c["window"] = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
            w = work(c)
            cells = c["batch"] * c["hq"] * c["new"] * c["ctx"]
            tokens = c["batch"] * c["hkv"] * c["dim"] * c["ctx"]
            if w["flops"] <= 1e11 and w["bytes"] <= 6e8 and cells <= 6e8 and tokens <= 3e8:
                return c


# ---------------------------------------------------------------------------
# what a case holds
# ---------------------------------------------------------------------------

def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence: ragged, the first one at the case's own
    sizes; the same for every seed, so that the work is the case's."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new, ctx = [case["new"]], [max(case["ctx"], case["new"])]
    for _ in range(case["batch"] - 1):
        n = case["new"] if case["new"] <= 8 else r.randint(max(1, case["new"] // 4), case["new"])
        new.append(n)
        ctx.append(max(n, r.randint(max(1, case["ctx"] // 4), case["ctx"])))
    return new, ctx


def _visible(first, last, window):
    """Keys that the queries at positions first .. last see, summed over the queries."""
    if window <= 0:
        return (first + last + 2) * (last - first + 1) // 2
    return sum(min(p + 1, window) for p in range(first, last + 1))


def work(case):
    size = SIZES[case["dtype"]]
    if case["op"] == "sample":
        cells = case["batch"] * case["vocab"]
        return {"bytes": cells * size + case["batch"] * 24, "flops": 4 * cells}
    new, ctx = _lengths(case)
    hq, hkv, dim, page = case["hq"], case["hkv"], case["dim"], case["page"]
    tokens = sum(new)
    if case["op"] == "append":
        # q in and out; k and v in, and their codes out
        bytes_ = tokens * dim * (2 * hq * size + 2 * hkv * (size + 1))
        return {"bytes": bytes_, "flops": tokens * 3 * case["rot"] * (hq + hkv) + tokens * hkv * dim * 4}
    pairs = read = 0
    for n, c in zip(new, ctx):
        pairs += _visible(c - n, c - 1, case["window"])
        read += c if case["window"] <= 0 else min(c, n + case["window"] - 1)
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


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "sample":
        batch, vocab, filters = case["batch"], case["vocab"], case["filters"]
        logits = (torch.randn(batch, vocab, device=DEV, generator=g) * 2.5).to(dtype)
        # a few tokens stand out, as in a trained model's logits
        top = torch.randint(0, vocab, (batch, 8), device=DEV, generator=g)
        logits.scatter_(1, top, (logits.gather(1, top).float().abs() + 8).to(dtype))
        s = {"case": case, "logits": logits, "u": torch.rand(batch, device=DEV, generator=g)}
        on = torch.rand(4, batch, device=DEV, generator=g) < (0.6 if filters == "mixed" else 2.0)
        pick = lambda lo, hi: torch.rand(batch, device=DEV, generator=g) * (hi - lo) + lo  # noqa: E731
        s["temperature"] = torch.where(on[0], pick(0.5, 1.3), torch.tensor(1.0, device=DEV))
        s["top_k"] = s["top_p"] = s["min_p"] = None
        if filters in ("top_k", "all", "mixed"):
            s["top_k"] = torch.where(on[1], pick(5, 200).int(), 0).int()
        if filters in ("top_p", "all", "mixed"):
            s["top_p"] = torch.where(on[2], pick(0.5, 0.98), torch.tensor(1.0, device=DEV))
        if filters in ("min_p", "all", "mixed"):
            s["min_p"] = torch.where(on[3], pick(0.005, 0.1), torch.tensor(0.0, device=DEV))
        return s
    new, ctx = _lengths(case)
    page, tokens = case["page"], sum(new)
    width = -(-max(ctx) // page)
    table = torch.full((len(new), width), -1, dtype=torch.int32)
    # the pages that the call reads or writes are the sequence's own; for an append, what lies before them stays elsewhere
    own_pages = [(((c - n) // page if case["op"] == "append" else 0), -(-c // page)) for n, c in zip(new, ctx)]
    pages = sum(b - a for a, b in own_pages)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).int()
    at = 0
    for i, (a, b) in enumerate(own_pages):
        table[i, a:b] = order[at:at + b - a]
        at += b - a
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    s = {"case": case, "cache": _cache(case, pages, g), "table": table.to(DEV),
         "lens": torch.tensor(ctx, dtype=torch.int32, device=DEV), "max_new": max(new),
         "cu": torch.tensor([0] + [sum(new[:i + 1]) for i in range(len(new))], dtype=torch.int32, device=DEV)}
    # q, k and v are the parts of one projection's rows
    qkv = torch.randn(tokens, (hq + 2 * hkv) * dim, device=DEV, generator=g).to(dtype)
    q, k, v = qkv.split([hq * dim, hkv * dim, hkv * dim], dim=1)
    s["q"] = q.unflatten(1, (hq, dim))
    if case["op"] == "append":
        s["k"], s["v"] = k.unflatten(1, (hkv, dim)), v.unflatten(1, (hkv, dim))
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV).float() / case["rot"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _append_outputs(s, q):
    c = s["cache"]
    return {"q": q, "k": c["k"].view(torch.float8_e4m3fn), "v": c["v"].view(torch.float8_e4m3fn),
            "k_scales": c["k_scales"], "v_scales": c["v_scales"]}


def _own_append(s):
    import nvfp4_quantized_matmul_amd as nv
    q = nv.kv_append(s["k"], s["v"], nv.KVCache(**s["cache"]), s["table"], s["lens"], q=s["q"], cu_q=s["cu"], max_q=s["max_new"],
                     inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"])
    return _append_outputs(s, q)


def _own_attention(s):
    import nvfp4_quantized_matmul_amd as nv
    return nv.paged_attention(s["q"], nv.KVCache(**s["cache"]), s["table"], s["lens"], cu_q=s["cu"], max_q=s["max_new"],
                              window=s["case"]["window"])


def _own_sample(s):
    import nvfp4_quantized_matmul_amd as nv
    return nv.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                     min_p=s["min_p"], return_prob=True)


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


def _rotate(x, cos, sin, interleaved):
    r = 2 * cos.shape[1]
    x = x.double()
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _plain_append(s):
    case, cache = s["case"], s["cache"]
    page = case["page"]
    cu, lens, table = s["cu"].long(), s["lens"].long(), s["table"].long()
    _, pos = _token_places(s)
    angle = pos[:, None].double() * s["inv_freq"].double()
    cos, sin = angle.cos(), angle.sin()
    q = _rotate(s["q"], cos, sin, case["interleaved"]).float().to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, case["interleaved"]).float()
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
    return _append_outputs(s, q)


def _plain_attention(s):
    case, cache = s["case"], s["cache"]
    hkv, dim, page = case["hkv"], case["dim"], case["page"]
    group = case["hq"] // hkv
    q, cu, lens = s["q"], s["cu"].long(), s["lens"].long()
    batch, width = s["table"].shape
    most = s["max_new"]
    # rows of each sequence beside each other: [sequences, kv heads, tokens * group, dim]
    t = torch.arange(most, device=DEV)
    count = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + t).clamp(0, q.shape[0] - 1)
    rows = q.float()[row].view(batch, most, hkv, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, hkv, -1, dim)
    ids = s["table"].long()
    there = ids >= 0
    ids = ids.clamp_min(0)

    def values(codes, scales):
        x = cache[codes][ids].view(torch.float8_e4m3fn).float()
        return x * torch.exp2(cache[scales][ids].float() - 127)[..., None, None]

    k = values("k", "k_scales").permute(0, 2, 1, 3, 4).reshape(batch, hkv, width * page, dim)
    at = torch.arange(width * page, device=DEV)
    pos = lens[:, None] - count[:, None] + t
    see = (at <= pos[..., None]) & there.repeat_interleave(page, 1)[:, None]
    if case["window"] > 0:
        see &= at > pos[..., None] - case["window"]
    see = see.repeat_interleave(group, 1)[:, None]
    score = torch.matmul(rows, k.transpose(2, 3)) * dim ** -0.5
    score = torch.where(see, score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top.isfinite(), top, 0.0))
    del score
    v = values("v", "v_scales").permute(0, 2, 1, 4, 3).reshape(batch, hkv, width * page, dim)
    v = torch.where((at < lens[:, None])[:, None, :, None], v, 0.0)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v) / torch.where(total > 0, total, 1.0)
    out = out.view(batch, hkv, most, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, most, hkv * group, dim)
    seq, at = _token_places(s)
    return out[seq, at - (lens - count)[seq]].to(q.dtype)


def _plain_sample(s):
    x = s["logits"].double()
    x = torch.where(x.isnan(), float("-inf"), x)
    batch, vocab = x.shape
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((x - x[:, :1]) / s["temperature"].double()[:, None])
    w = torch.where(x == x[:, :1], 1.0, w)
    w = torch.where(x == float("-inf"), 0.0, w)
    rank = torch.arange(vocab, device=DEV)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        w = torch.where((rank < k) | (k <= 0), w, 0.0)
    keep = w > 0
    if s["top_p"] is not None:
        before = w.cumsum(1) - w
        keep &= before < s["top_p"].double()[:, None] * w.sum(1, keepdim=True)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    w = torch.where(keep | ((rank == 0) & (w > 0)), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)
    c = w.cumsum(1)
    token = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(1)
    some = c[:, -1] > 0
    prob = w.gather(1, token.clamp_max(vocab - 1)[:, None])[:, 0] / torch.where(some, c[:, -1], 1.0)
    return torch.where(some, token, -1).int(), prob.float()


_PLAIN = {"append": _plain_append, "attention": _plain_attention, "sample": _plain_sample}
_OWN = {"append": _own_append, "attention": _own_attention, "sample": _own_sample}


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
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](s)


def _exact_append(s):
    case, cache, page = s["case"], s["cache"], s["case"]["page"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    e4m3 = _e4m3_table()
    half = case["rot"] // 2
    freq = s["inv_freq"].double()
    lane = torch.arange(half, device=DEV)
    ia, ib = (2 * lane, 2 * lane + 1) if case["interleaved"] else (lane, lane + half)
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    codes = {n: e4m3[cache[n].int()] for n in ("k", "v")}
    bytes_ = {n: cache[n + "_scales"].int() for n in ("k", "v")}
    for b in range(len(lens)):
        lo, hi = cu[b], cu[b + 1]
        first = lens[b] - (hi - lo)
        turn = torch.outer(torch.arange(first, lens[b], device=DEV, dtype=torch.float64), freq)
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
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    e4m3 = _e4m3_table()
    q = s["q"].double()
    out = torch.zeros_like(q)
    group = case["hq"] // case["hkv"]
    for b in range(len(lens)):
        lo, hi, n = cu[b], cu[b + 1], lens[b]
        ids = s["table"][b, :-(-n // page)].long()
        pos = torch.arange(n - (hi - lo), n, device=DEV)
        at = torch.arange(n, device=DEV)
        hidden = at[None] > pos[:, None]
        if case["window"] > 0:
            hidden |= at[None] <= pos[:, None] - case["window"]
        for h in range(case["hkv"]):
            k = e4m3[cache["k"][ids, h].int()] * torch.exp2(cache["k_scales"][ids, h].double() - 127)[:, None, None]
            v = e4m3[cache["v"][ids, h].int()] * torch.exp2(cache["v_scales"][ids, h].double() - 127)[:, None, None]
            k, v = k.reshape(-1, case["dim"])[:n], v.transpose(1, 2).reshape(-1, case["dim"])[:n]
            for j in range(h * group, (h + 1) * group):
                z = (q[lo:hi, j] @ k.T / math.sqrt(case["dim"])).masked_fill_(hidden, float("-inf"))
                out[lo:hi, j] = torch.softmax(z, 1) @ v
    return out


def _exact_sample(s):
    """The probabilities, row by row on the host; the token numbers have to be equal and are not here."""
    get = lambda name, i, default: default if s[name] is None else s[name][i].item()  # noqa: E731
    prob = []
    for i, row in enumerate(s["logits"].double().cpu()):
        w = torch.exp((row - row.max()) / get("temperature", i, 1.0))
        order = torch.argsort(row, descending=True, stable=True)
        k = get("top_k", i, 0)
        order = order[:k] if k > 0 else order
        mass = torch.cat((torch.zeros(1, dtype=torch.float64), w[order].cumsum(0)))
        order = order[:int((mass[:-1] < get("top_p", i, 1.0) * mass[-1]).sum())]
        order = order[w[order] >= get("min_p", i, 0.0)]
        kept = torch.sort(order).values
        c = w[kept].cumsum(0)
        at = min(int(torch.searchsorted(c, s["u"][i].item() * c[-1].item(), right=True)), len(kept) - 1)
        prob.append(w[kept[at]] / c[-1])
    return None, torch.stack(prob)
