"""Cases of the paged serving operators: page tables and slot maps, K/V append,
and attention of new tokens over the paged cache.

Each case names one call of one operator.  `run` computes it in elementary
torch operations, or with `own` set by the library's entry points.
"""
import math
import random

import torch

own = False  # True: run() calls the library

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of a full serving batch: one new token per request,
        # a new page for about one request in 64.  Latency is what counts.
        {"name": "pages_decode", "op": "pages", "seqs": 256, "q_min": 1, "q_max": 1,
         "ctx_min": 100, "ctx_max": 32768, "page": 64, "lens": 1},
        # A step of prompt chunks: ragged chunks over ragged contexts.
        {"name": "pages_chunks", "op": "pages", "seqs": 512, "q_min": 16, "q_max": 1024,
         "ctx_min": 0, "ctx_max": 65536, "page": 64, "lens": 2},
        # Requests that ended or rolled back give their pages back.
        {"name": "pages_release", "op": "release", "seqs": 1000, "ctx_min": 1, "ctx_max": 8192,
         "page": 16, "lens": 3},
        # The decode step's new K and V rows, views of a fused QKV projection.
        {"name": "append_decode", "op": "append", "tokens": 256, "q_heads": 64, "kv_heads": 8,
         "dim": 128, "page": 64, "dtype": "bf16"},
        # A whole 128K prompt's K and V rows.
        {"name": "append_prompt", "op": "append", "tokens": 131072, "q_heads": 64, "kv_heads": 8,
         "dim": 128, "page": 64, "dtype": "bf16"},
        # A small decode step: four requests with short contexts.
        {"name": "step_small", "op": "attend", "seqs": 4, "q_min": 1, "q_max": 1, "ctx_min": 300,
         "ctx_max": 2047, "q_heads": 32, "kv_heads": 4, "dim": 128, "page": 64, "window": 0,
         "causal": True, "dtype": "bf16", "lens": 4},
        # A decode step of a full batch over ragged contexts up to 32K.
        {"name": "step_batch", "op": "attend", "seqs": 64, "q_min": 1, "q_max": 1, "ctx_min": 500,
         "ctx_max": 32767, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "window": 0,
         "causal": True, "dtype": "bf16", "lens": 5},
        # One decode step at the end of a context of 1M tokens.
        {"name": "step_1m", "op": "attend", "seqs": 1, "q_min": 1, "q_max": 1, "ctx_min": 1048575,
         "ctx_max": 1048575, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "window": 0,
         "causal": True, "dtype": "bf16", "lens": 6},
        # Chunked prefill: 4096 new tokens behind 32K cached ones.
        {"name": "chunk_32k", "op": "attend", "seqs": 1, "q_min": 4096, "q_max": 4096,
         "ctx_min": 32768, "ctx_max": 32768, "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64,
         "window": 0, "causal": True, "dtype": "bf16", "lens": 7},
        # A mixed step: ragged chunks and single tokens in one call, small pages.
        {"name": "chunk_mixed", "op": "attend", "seqs": 9, "q_min": 1, "q_max": 501, "ctx_min": 600,
         "ctx_max": 9001, "q_heads": 32, "kv_heads": 4, "dim": 128, "page": 16, "window": 0,
         "causal": True, "dtype": "bf16", "lens": 8},
        # A sliding-window layer on prompts that are new or partly cached.
        {"name": "chunk_window", "op": "attend", "seqs": 4, "q_min": 1500, "q_max": 8192,
         "ctx_min": 0, "ctx_max": 4096, "q_heads": 32, "kv_heads": 4, "dim": 64, "page": 32,
         "window": 512, "causal": True, "dtype": "bf16", "lens": 9},
        # fp32 cache, one KV head: the precision a reference run is made in.
        {"name": "chunk_fp32", "op": "attend", "seqs": 3, "q_min": 100, "q_max": 401,
         "ctx_min": 0, "ctx_max": 1701, "q_heads": 4, "kv_heads": 1, "dim": 64, "page": 8,
         "window": 0, "causal": True, "dtype": "fp32", "lens": 10},
    ]


MOST_BYTES = 9e9   # about the largest listed cases' work
MOST_FLOPS = 4.7e12
MOST_SCORES = 9e9  # padded score values of the plain form


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    lens = rng.randrange(1 << 30)
    op = rng.choice(["pages", "release", "append", "attend", "attend", "attend", "attend"])
    page = rng.choice([8, 16, 24, 32, 64, 64, 128])
    if op == "pages":
        q_max = rng.choice([1, 1, _log(rng, 2, 2048)])
        ctx = _log(rng, 16, 131072)
        return {"op": op, "seqs": _log(rng, 1, 600), "q_min": 1, "q_max": q_max,
                "ctx_min": rng.choice([0, ctx // 3]), "ctx_max": ctx, "page": page, "lens": lens}
    if op == "release":
        return {"op": op, "seqs": _log(rng, 1, 2000), "ctx_min": 1, "ctx_max": _log(rng, 16, 16384),
                "page": page, "lens": lens}
    heads = rng.choice([(64, 8, 128), (32, 4, 128), (32, 4, 64), (4, 1, 64), (28, 4, 128),
                        (8, 8, 64), (8, 1, 128)])
    shape = {"q_heads": heads[0], "kv_heads": heads[1], "dim": heads[2], "page": page}
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 60000), **shape, "dtype": dtype}
    while True:
        q_max = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 4096)])
        ctx = _log(rng, 64, 65536 if dtype == "bf16" else 4096)
        c = {"op": op, "seqs": _log(rng, 1, 64), "q_min": rng.choice([1, q_max]), "q_max": q_max,
             "ctx_min": rng.choice([0, ctx // 2, ctx]), "ctx_max": ctx, **shape,
             "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)]), "causal": True, "dtype": dtype,
             "lens": lens}
        if not c["window"]:
            c["causal"] = rng.random() < 0.9
        w = work(c)
        most = MOST_FLOPS if dtype == "bf16" else MOST_FLOPS / 20
        scores = c["seqs"] * c["q_heads"] * q_max * (ctx + q_max)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= most and scores <= MOST_SCORES:
            return c


def _lengths(case):
    """(new tokens, cache length after the step) of each sequence: the case's
    own ragged lengths, the first sequence at the range's upper end and the
    last one (of more than eight, with chunks) idle."""
    r = random.Random(case["lens"])
    n = case["seqs"]
    q_min, q_max = case.get("q_min", 0), case.get("q_max", 0)
    q = [q_max if i == 0 else _log(r, max(1, q_min), max(1, q_max)) if q_max else 0
         for i in range(n)]
    ctx = [case["ctx_max"] if i == 0 else _log(r, case["ctx_min"] + 1, case["ctx_max"] + 1) - 1
           for i in range(n)]
    if q_max > 1 and n > 8:
        q[-1] = 0
    return q, [a + b for a, b in zip(q, ctx)]


def _pages(length, page):
    return (length + page - 1) // page


def _visible(pos, kv, window, causal):
    """Keys that the query at `pos` sees."""
    hi = min(kv, pos + 1) if causal else kv
    lo = max(0, pos + 1 - window) if window else 0
    return max(0, hi - lo)


def work(case):
    op = case["op"]
    if op == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["tokens"] * (8 + 4 * case["kv_heads"] * case["dim"] * e), "flops": 0}
    q, kv = _lengths(case)
    page = case["page"]
    if op == "pages":
        new = sum(_pages(b, page) - _pages(b - a, page) for a, b in zip(q, kv))
        return {"bytes": 16 * len(q) + 8 * new + 12 * sum(q), "flops": 0}
    if op == "release":
        back = sum(_pages(b, page) - _pages(k, page) for b, k in zip(kv, _kept(case, kv)))
        return {"bytes": 8 * len(kv) + 8 * back, "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    d, hq, hk = case["dim"], case["q_heads"], case["kv_heads"]
    rows, keys, pairs = sum(q), 0, 0
    for a, b in zip(q, kv):
        if a == 0:
            continue
        first = _visible(b - a, b, case["window"], case["causal"])
        keys += min(b, first + a - 1 if case["window"] else b)
        if not case["causal"]:
            pairs += a * b
        elif not case["window"]:
            pairs += a * (b - a) + a * (a + 1) // 2
        else:
            pairs += sum(_visible(b - a + i, b, case["window"], True) for i in range(a))
    return {"bytes": rows * hq * (2 * d * e + 4) + 2 * keys * hk * d * e + 4 * len(q),
            "flops": 4.0 * d * hq * pairs}


def _kept(case, kv):
    """What each request keeps: nothing when it ended (three in four), else a
    prefix (drafted tokens that were not accepted are taken back)."""
    r = random.Random(case["lens"] + 1)
    return [0 if r.random() < 0.75 else max(0, n - r.randint(0, 64)) for n in kv]


# -------------------------------------------------------------------- inputs
def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    op, page = case["op"], case["page"]
    s["status"] = torch.zeros(4, dtype=torch.int32, device=DEV)
    if op == "append":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        n_pages = _pages(t, page) + 7
        qkv = torch.randn(t, (hq + 2 * hk) * d, device=DEV, generator=g).to(DTYPES[case["dtype"]])
        s["K"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["V"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        # new rows come in page order: each page of a random permutation in turn
        order = torch.randperm(n_pages, device=DEV, generator=g)
        at = torch.arange(t, device=DEV) + 3
        s["slot_map"] = order[at // page] * page + at % page
        s["K_pages"] = torch.zeros(n_pages, hk, page, d, dtype=qkv.dtype, device=DEV)
        s["V_pages"] = torch.zeros_like(s["K_pages"])
        s["n_pages"] = n_pages
        return s
    q, kv = _lengths(case)
    s["seqs"], s["max_pages"] = len(q), max(1, max(_pages(n, page) for n in kv))
    s["total"] = sum(q)
    s["q_len"], s["kv_len"] = _int(q), _int(kv)
    held = [_pages(b - (a if op == "pages" else 0), page) for a, b in zip(q, kv)]
    after = [_pages(b, page) for b in kv]
    s["n_pages"] = sum(after) + 5
    order = torch.randperm(s["n_pages"], device=DEV, generator=g).to(torch.int32)
    # rows of the page table: the pages each sequence holds, -1 behind them
    table = torch.full((len(q), s["max_pages"]), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(s["max_pages"], device=DEV)
    inside = col[None, :] < _int(held)[:, None]
    table[inside] = order[:sum(held)]
    s["page_table"] = table
    if op in ("pages", "release"):
        free = s["n_pages"] - sum(held)
        stack = torch.full((s["n_pages"],), -1, dtype=torch.int32, device=DEV)
        stack[:free] = order[sum(held):]
        s["free_pages"], s["n_free"] = stack, _int([free])
        s["n_free_out"] = torch.zeros_like(s["n_free"])
        s["q_start"] = torch.zeros(len(q) + 1, dtype=torch.int32, device=DEV)
        s["slot_map"] = torch.zeros(s["total"], dtype=torch.int64, device=DEV)
        s["positions"] = torch.zeros(s["total"], dtype=torch.int32, device=DEV)
        if op == "release":
            s["keep_len"] = _int(_kept(case, kv))
        return s
    hq, hk, d, dt = case["q_heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    s["q_start"] = _int([sum(q[:i]) for i in range(len(q) + 1)])
    s["max_q"], s["max_kv"] = max(q), max(kv)
    # logits of standard deviation 2: neither flat nor a single winner
    s["Q"] = (2 * torch.randn(s["total"], hq, d, device=DEV, generator=g)).to(dt)
    shape = (s["n_pages"], hk, page, d)
    s["K_pages"] = torch.empty(shape, dtype=dt, device=DEV).normal_(generator=g)
    s["V_pages"] = torch.empty(shape, dtype=dt, device=DEV).normal_(generator=g)
    s["O"] = torch.zeros_like(s["Q"])
    s["lse"] = torch.zeros(hq, s["total"], dtype=torch.float32, device=DEV)
    return s


# --------------------------------------------------------------- plain forms
def _plain_pages(s):
    page, q, kv = s["page"], s["q_len"].long(), s["kv_len"].long()
    held, after = (kv - q + page - 1) // page, (kv + page - 1) // page
    need = after - held
    ends = need.cumsum(0)
    n_free = s["n_free"].long()
    col = torch.arange(s["max_pages"], device=DEV)
    new = (col >= held[:, None]) & (col < after[:, None])
    take = n_free - 1 - ((ends - need)[:, None] + col - held[:, None])
    table = torch.where(new, s["free_pages"][take.clamp(0, s["n_pages"] - 1)], s["page_table"])
    q_start = torch.cat([q.new_zeros(1), q.cumsum(0)])
    t = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(q_start[1:], t, right=True)
    pos = (kv - q)[seq] + t - q_start[seq]
    slot = table[seq, pos // page].long() * page + pos % page
    return {"page_table": table, "q_start": q_start.int(), "slot_map": slot,
            "positions": pos.int(), "n_free": (n_free - ends[-1]).int()}


def _plain_release(s):
    page, n_pages = s["page"], s["n_pages"]
    keep, held = (s["keep_len"].long() + page - 1) // page, (s["kv_len"].long() + page - 1) // page
    back = held - keep
    ends = back.cumsum(0)
    n_free = s["n_free"].long()
    col = torch.arange(s["max_pages"], device=DEV)
    ours = (col >= keep[:, None]) & (col < held[:, None])
    at = n_free + (ends - back)[:, None] + col - keep[:, None]
    at = torch.where(ours, at, n_pages)  # one place behind the stack takes the rest
    stack = torch.cat([s["free_pages"], s["free_pages"][:1]])
    stack = stack.scatter(0, at.flatten(), s["page_table"].flatten())[:n_pages]
    return {"free_pages": stack, "n_free": (n_free + ends[-1]).int()}


def _plain_append(s):
    page, off = s["slot_map"] // s["page"], s["slot_map"] % s["page"]
    s["K_pages"][page, :, off] = s["K"]
    s["V_pages"][page, :, off] = s["V"]
    return {"K_pages": s["K_pages"], "V_pages": s["V_pages"]}


def _plain_attend(s):
    n, page, d = s["seqs"], s["page"], s["dim"]
    hk, group = s["kv_heads"], s["q_heads"] // s["kv_heads"]
    q_start, kv = s["q_start"].long(), s["kv_len"].long()
    q_len = q_start[1:] - q_start[:-1]
    key, row = torch.arange(s["max_kv"], device=DEV), torch.arange(s["max_q"], device=DEV)
    pages = s["page_table"].long().clamp(min=0)[:, key // page]
    q = s["Q"][(q_start[:-1, None] + row).clamp(max=s["total"] - 1)].float()
    q = q.unflatten(2, (hk, group)).transpose(1, 2).reshape(n, hk, -1, d)
    k = s["K_pages"][pages, :, key % page].float()
    score = q @ k.permute(0, 2, 3, 1)
    del k
    score = score.mul_(1 / math.sqrt(d)).view(n, hk, s["max_q"], group, s["max_kv"])
    pos = ((kv - q_len)[:, None] + row)[:, None, :, None, None]
    seen = key < kv[:, None, None, None, None]
    if s["causal"]:
        seen = seen & (key <= pos)
    if s["window"]:
        seen = seen & (key > pos - s["window"])
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top.clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = score.sum(-1, keepdim=True)
    v = s["V_pages"][pages, :, key % page].float().permute(0, 2, 1, 3)
    o = (score.flatten(2, 3) @ v).view(n, hk, s["max_q"], group, d)
    o = o / total.masked_fill(total == 0, 1)
    lse = (top + total.log()).squeeze(-1)
    t = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(q_start[1:], t, right=True)
    at = t - q_start[seq]
    return {"O": o[seq, :, at].flatten(1, 2).to(s["Q"].dtype),
            "lse": lse[seq, :, at].flatten(1, 2).t()}


# ------------------------------------------------------------ the library's
def _handle(s, sgqa):
    """The parameters and workspace that a serving loop keeps between steps."""
    if "params" not in s:
        s["params"] = sgqa.paged_params(
            n_seqs=s.get("seqs", 0), max_tokens=s.get("total", s.get("tokens")),
            n_q_heads=s.get("q_heads", 1), n_kv_heads=s.get("kv_heads", 1),
            head_dim=s.get("dim", 64), page_size=s["page"], n_pages=s["n_pages"],
            max_pages=s.get("max_pages", 1),
            dtype=sgqa.FP32 if s.get("dtype") == "fp32" else sgqa.BF16,
            causal=s.get("causal", True), window=s.get("window", 0),
            kv_stride=s["K"].stride(0) if "K" in s else 0)
        if s["op"] == "attend":
            s["ws"] = sgqa.alloc_paged_workspace(s["params"], DEV)
    return s["params"]


def _own(s):
    from block_sparse_long_sgqa_gb300 import sgqa

    p = _handle(s, sgqa)
    if s["op"] == "pages":
        sgqa.sgqa_page_plan(p, s["q_len"], s["kv_len"], s["free_pages"], s["n_free"],
                            s["page_table"], s["q_start"], s["slot_map"], s["positions"],
                            s["n_free_out"], status=s["status"])
        return {"page_table": s["page_table"], "q_start": s["q_start"],
                "slot_map": s["slot_map"], "positions": s["positions"], "n_free": s["n_free_out"]}
    if s["op"] == "release":
        sgqa.sgqa_page_release(p, s["kv_len"], s["keep_len"], s["page_table"], s["free_pages"],
                               s["n_free"], s["n_free_out"], status=s["status"])
        return {"free_pages": s["free_pages"], "n_free": s["n_free_out"]}
    if s["op"] == "append":
        sgqa.sgqa_paged_append(p, s["K"], s["V"], s["slot_map"], s["K_pages"], s["V_pages"],
                               status=s["status"])
        return {"K_pages": s["K_pages"], "V_pages": s["V_pages"]}
    sgqa.sgqa_paged_attn(p, s["Q"], s["K_pages"], s["V_pages"], s["page_table"], s["q_start"],
                         s["kv_len"], s["O"], s["lse"], s["ws"], status=s["status"])
    return {"O": s["O"], "lse": s["lse"]}


PLAIN = {"pages": _plain_pages, "release": _plain_release, "append": _plain_append,
         "attend": _plain_attend}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# --------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """Attention by its definition, a sequence and a KV head at a time; the
    appended pools as rows of a flat cache.  Page tables hold no computed
    floating values."""
    if case["op"] in ("pages", "release") or work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "append":
        out = {}
        for name in ("K", "V"):
            pool = s[name + "_pages"].double().transpose(1, 2).flatten(0, 1).contiguous()
            pool.index_copy_(0, s["slot_map"], s[name].double())
            out[name + "_pages"] = pool.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
        return out
    q_len, kv_len = _lengths(case)
    group = case["q_heads"] // case["kv_heads"]
    o = torch.zeros(s["Q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for i, (a, b) in enumerate(zip(q_len, kv_len)):
        ids = s["page_table"][i, :_pages(b, page)].long()
        for g in range(case["kv_heads"] if a and b else 0):
            k = s["K_pages"][ids, g].flatten(0, 1)[:b].double()
            v = s["V_pages"][ids, g].flatten(0, 1)[:b].double()
            for h in range(g * group, (g + 1) * group):
                x = s["Q"][first:first + a, h].double() @ k.t() / math.sqrt(case["dim"])
                p = torch.arange(b - a, b, device=DEV)[:, None]
                j = torch.arange(b, device=DEV)[None, :]
                if case["causal"]:
                    x[(j > p).expand_as(x)] = -math.inf
                if case["window"]:
                    x[(j <= p - case["window"]).expand_as(x)] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[h, first:first + a] = z
                x.sub_(z[:, None].clamp(min=-1e300)).exp_()
                o[first:first + a, h] = x @ v
        first += a
    return {"O": o, "lse": lse}
