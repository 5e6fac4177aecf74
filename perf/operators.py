"""What the K/V-cache operators are measured on: appending to a paged 8-bit cache, attention over it, attention of
prompts through a sliding window with sinks, and the management of the cache's pages."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # a batch of prompts enters the cache
        {"name": "append-prompts", "op": "append", "B": 8, "L": 4096, "kv_heads": 8, "dim": 128, "page": 64, "held": 0,
         "dtype": "bf16"},
        # one decode step of a batch: a token for each sequence, most of them into a page that is partly full
        {"name": "append-step", "op": "append", "B": 256, "L": 1, "kv_heads": 8, "dim": 128, "page": 64, "held": 2000,
         "dtype": "bf16"},
        # a single user's decode step over a short context: latency
        {"name": "attend-one", "op": "attend", "B": 1, "L": 1, "heads": 64, "kv_heads": 8, "dim": 128, "page": 16,
         "tokens": 500, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a decode step of a serving batch with contexts of different lengths
        {"name": "attend-batch", "op": "attend", "B": 64, "L": 1, "heads": 64, "kv_heads": 8, "dim": 128, "page": 64,
         "tokens": 8192, "window": 0, "sinks": 0, "dtype": "bf16"},
        # one long context whose 64 query heads share one key/value head
        {"name": "attend-long", "op": "attend", "B": 1, "L": 1, "heads": 64, "kv_heads": 1, "dim": 128, "page": 128,
         "tokens": 262143, "window": 0, "sinks": 0, "dtype": "bf16"},
        # drafted tokens checked four at a time, narrow heads
        {"name": "attend-draft", "op": "attend", "B": 16, "L": 4, "heads": 32, "kv_heads": 8, "dim": 64, "page": 32,
         "tokens": 16384, "window": 0, "sinks": 0, "dtype": "fp16"},
        # a decode step of the window branch: 128 tokens and the sinks of each sequence
        {"name": "attend-window", "op": "attend", "B": 128, "L": 1, "heads": 64, "kv_heads": 8, "dim": 128, "page": 16,
         "tokens": 4096, "window": 128, "sinks": 4, "dtype": "bf16"},
        # two short prompts without shared heads
        {"name": "window-short", "op": "window", "B": 2, "S": 777, "heads": 16, "kv_heads": 16, "dim": 64,
         "window": 128, "sinks": 0, "dtype": "fp16"},
        # a long prompt of the window branch
        {"name": "window-prompt", "op": "window", "B": 1, "S": 16384, "heads": 64, "kv_heads": 8, "dim": 128,
         "window": 128, "sinks": 4, "dtype": "bf16"},
        # padded prompts with a wide window
        {"name": "window-wide", "op": "window", "B": 2, "S": 8192, "heads": 32, "kv_heads": 4, "dim": 128,
         "window": 2048, "sinks": 16, "dtype": "bf16"},
        # parallel samples: each prompt forked eight times, then room for the next tokens
        {"name": "pages-fork", "op": "fork", "rows": 64, "forks": 8, "tokens": 2000, "extra": 64, "share": True,
         "kv_heads": 8, "dim": 128, "page": 64},
        # finished sequences leave, and the rest moves together
        {"name": "pages-compact", "op": "compact", "rows": 128, "tokens": 4096, "kv_heads": 8, "dim": 128, "page": 64},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attend", "attend", "window", "window", "fork", "compact"])
    c = {"op": op, "dim": rng.choice([64, 128])}
    if op == "append":
        c |= {"kv_heads": rng.randint(1, 8), "page": rng.choice([16, 32, 64, 128]), "held": rng.choice([0, log(1, 4000)]),
              "dtype": rng.choice(["bf16", "fp16"])}
        c["L"] = log(1, 4096)
        c["B"] = log(1, max(1, min(256, 32768 // c["L"])))
    elif op == "attend":
        c |= {"kv_heads": rng.randint(1, 8), "page": rng.choice([16, 32, 64, 128]), "L": rng.choice([1, 1, 2, 3, 4]),
              "window": rng.choice([0, 0, log(16, 4096)]), "dtype": rng.choice(["bf16", "fp16"])}
        c["sinks"] = rng.randint(1, 64) if c["window"] and rng.random() < 0.5 else 0
        c["heads"] = c["kv_heads"] * log(1, 64 // c["kv_heads"])
        c["tokens"] = log(4, 262144)
        c["B"] = log(1, max(1, min(128, (1 << 21) // (c["tokens"] * c["kv_heads"]))))
    elif op == "window":
        c |= {"kv_heads": rng.randint(1, 8), "window": log(1, 2048), "sinks": rng.choice([0, rng.randint(1, 64)]),
              "dtype": rng.choice(["bf16", "fp16"]), "S": log(1, 16384)}
        c["heads"] = c["kv_heads"] * log(1, 64 // c["kv_heads"])
        most = (1 << 29) // (c["S"] * c["heads"] * min(c["S"], c["window"] + 256))
        c["B"] = log(1, max(1, min(8, most)))
        while c["B"] * c["S"] * c["heads"] * min(c["S"], c["window"] + 256) > 1 << 30:
            c["S"] //= 2
    else:
        c |= {"kv_heads": rng.randint(1, 8), "page": rng.choice([16, 32, 64, 128]), "tokens": log(1, 4096)}
        c["rows"] = log(1, 64 if op == "fork" else 128)
        if op == "fork":
            c |= {"forks": log(1, 8), "extra": log(1, 256), "share": rng.random() < 0.7}
            if not c["share"]:
                c["forks"] = min(c["forks"], 2)
    return c


def spread(top, n):
    """n lengths of up to `top` tokens, the first the longest, none of them alike in earnest."""
    return [top - int(top * 0.5 * ((0.6180339887 * i) % 1.0)) for i in range(n)]


def lengths(case):
    """The lengths that a case's sequences have: the same for every seed, since the work depends on them."""
    if case["op"] == "append":
        held = [min(case["held"], h) for h in spread(case["held"], case["B"])]
        new = spread(case["L"], case["B"])
        return held, new
    if case["op"] == "attend":
        return spread(case["tokens"], case["B"])
    if case["op"] == "window":
        return spread(case["S"], case["B"])
    return spread(case["tokens"], case["rows"])


def pool(n_pages, case, g):
    """Pages as a cache holds them after a while: codes over the whole range, scales that differ by page and head."""
    def codes():
        shape = (n_pages, case["kv_heads"], case["page"], case["dim"])
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float16).mul_(96).clamp_(-448, 448).to(FP8)

    def scales():
        return torch.exp2(torch.randint(-8, -5, (n_pages, case["kv_heads"]), generator=g, device="cuda").float())

    return codes(), codes(), scales(), scales()


def tables(lens, rows, width, page, n_pages, g):
    """Page tables [rows, width] of sequences that hold `lens` tokens each, on shuffled pages; -1 where there is none."""
    need = torch.tensor([-(-x // page) for x in lens] + [0] * (rows - len(lens)), device="cuda")
    slot = torch.arange(width, device="cuda")
    has = slot < need[:, None]
    order = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    table[has] = order[: int(need.sum())]
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[has].long()] = 1
    return table, refs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(DTYPES[case["dtype"]])

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    op, page = case["op"], case.get("page")
    if op == "append":
        held, new = lengths(case)
        total = [a + b for a, b in zip(held, new)]
        width = -(-max(total) // page)
        n_pages = sum(-(-t // page) for t in total) + 1
        s["pool"] = pool(n_pages, case, g)
        s["table"], _ = tables(total, case["B"], width, page, n_pages, g)
        s["lens"], s["new"] = ints(held), ints(new)
        # key channels of different size, as projections give them
        size = torch.exp(torch.randn((case["kv_heads"], case["dim"]), generator=g, device="cuda"))
        s["k"] = (normal(case["B"], case["L"], case["kv_heads"], case["dim"]) * size).to(DTYPES[case["dtype"]])
        s["v"] = normal(case["B"], case["L"], case["kv_heads"], case["dim"])
    elif op == "attend":
        lens = lengths(case)
        n_pages = sum(-(-t // page) for t in lens) + 1
        s["pool"] = pool(n_pages, case, g)
        s["table"], _ = tables(lens, case["B"], -(-max(lens) // page), page, n_pages, g)
        s["lens"] = ints(lens)
        s["q"] = normal(case["B"], case["L"], case["heads"], case["dim"])
    elif op == "window":
        s["lens"] = ints(lengths(case))
        s["q"] = normal(case["B"], case["S"], case["heads"], case["dim"])
        s["k"] = normal(case["B"], case["S"], case["kv_heads"], case["dim"])
        s["v"] = normal(case["B"], case["S"], case["kv_heads"], case["dim"])
    else:
        lens = lengths(case)
        used = sum(-(-t // page) for t in lens)
        if op == "fork":
            children = case["rows"] * case["forks"]
            rows = case["rows"] + children
            n_pages = used + children * (2 if case["share"] else 1 + -(-max(lens) // page)) + children * -(-case["extra"] // page) + 7
            s["src"] = ints([i % case["rows"] for i in range(children)])
            s["dst"] = ints([case["rows"] + i for i in range(children)])
            width = -(-(max(lens) + case["extra"]) // page)
            s["new"] = ints([case["extra"]] * rows)
        else:
            rows, n_pages, width = case["rows"], used + 5, -(-max(lens) // page)
            gone = torch.randperm(rows, generator=g, device="cuda")[: (rows + 1) // 2]
            s["gone"] = gone.to(torch.int32).sort().values
        s["pool"] = pool(n_pages, case, g)
        table, refs = tables(lens, rows, width, page, n_pages, g)
        # one buffer, so that a pass can begin from the same state with one copy
        s["held"] = torch.cat([table.reshape(-1), ints(lens + [0] * (rows - len(lens))), refs])
        s["shape"] = (rows, width)
    return s


def state_of(s):
    """The tables, lengths and reference counts that a pass works on: a copy, since it changes them."""
    held = s["held"].clone()
    rows, width = s["shape"]
    return held[: rows * width].view(rows, width), held[rows * width: rows * (width + 1)], held[rows * (width + 1):]


def run(s):
    case = s["case"]
    if own:
        return run_own(s, case)
    return {"append": plain_append, "attend": plain_attend, "window": plain_window, "fork": plain_fork,
            "compact": plain_compact}[case["op"]](s, case)


def run_own(s, case):
    import streaming_top_b200 as si

    op = case["op"]
    if op == "window":
        return si.window_attention(s["q"], s["k"], s["v"], window=case["window"], n_sink=case["sinks"], lens=s["lens"])
    cache = si.PagedCache(*s["pool"])
    if op == "append":
        si.cache_append(cache, s["k"], s["v"], s["table"], s["lens"], n_new=s["new"])
        return s["pool"]
    if op == "attend":
        return si.cache_attention(s["q"], cache, s["table"], s["lens"], window=case["window"], n_sink=case["sinks"])
    table, lens, refs = state_of(s)
    if op == "fork":
        forked = si.cache_fork(cache, table, lens, refs, s["src"], s["dst"], share=case["share"])
        given = si.cache_reserve(cache, table, lens, refs, s["new"])
        return s["pool"], table, lens, refs, forked, given
    si.cache_free(cache, table, lens, refs, s["gone"])
    used, moved = si.cache_compact(cache, table, refs)
    return s["pool"], table, lens, refs, used, moved


# ---- the plain forms


def power_scale(amax):
    """The least power of two s with amax <= 448 s (0 for 0)."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875)).clamp(min=-126)), 0.0)


def encode(x, scale):
    return torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0).clamp(-448, 448).to(FP8)


def plain_append(s, case):
    page, B, L = case["page"], case["B"], case["L"]
    table, lens, new = s["table"].long(), s["lens"].long(), s["new"].long()
    i = torch.arange(L, device="cuda")
    at = lens[:, None] + i
    ok = i < new[:, None]
    n_pages = s["pool"][0].shape[0]
    into = torch.where(ok, table.gather(1, (at // page).clamp(max=table.shape[1] - 1)), n_pages)
    # the sequences that begin inside a page, and that page's older tokens
    part = (lens % page > 0) & (new > 0)
    first = table.gather(1, (lens // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    first = torch.where(part, first, n_pages)
    for codes, scales, rows in ((s["pool"][0], s["pool"][2], s["k"]), (s["pool"][1], s["pool"][3], s["v"])):
        x = rows.float()
        top = torch.zeros((n_pages + 1, case["kv_heads"]), device="cuda")
        amax = torch.where(ok[..., None], x.abs().amax(-1), 0.0)
        top.scatter_reduce_(0, into.reshape(-1, 1).expand(-1, case["kv_heads"]), amax.reshape(B * L, -1), "amax")
        scale = power_scale(top)
        padded = torch.cat([scales, scales.new_zeros(1, case["kv_heads"])])
        old = padded[first]
        scale[first] = torch.maximum(scale[first], old)
        bits = codes.view(torch.uint8)
        f = first.clamp(max=n_pages - 1)
        before = bits[f]
        value = before.view(FP8).float() * old[..., None, None]
        again = encode(value, scale[first][..., None, None].expand_as(value)).view(torch.uint8)
        older = (torch.arange(page, device="cuda") < (lens % page)[:, None])[:, None, :, None] & part[:, None, None, None]
        keep = part.nonzero()[:, 0]
        bits[f[keep]] = torch.where(older, again, before)[keep]
        code = encode(x, scale[into][..., None].expand_as(x)).view(torch.uint8)
        b, t = ok.nonzero(as_tuple=True)
        bits[into[b, t], :, at[b, t] % page] = code[b, t]
        touched = into[b, t]
        scales[touched] = scale[touched]
    return s["pool"]


def visible(pos, key, case):
    """Whether the query at `pos` sees the key at `key`."""
    see = (key <= pos) & (key >= 0)
    if case["window"]:
        see = see & ((key > pos - case["window"]) | (key < case["sinks"]))
    return see


def softmax_parts(scores, see):
    """(weights, lse) of scores masked by `see` along the last axis; rows that see nothing get zeros and -inf."""
    scores = scores.masked_fill(~see, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0), (torch.log(total) + top)[..., 0]


def plain_attend(s, case):
    B, L, H, G, D = case["B"], case["L"], case["heads"], case["kv_heads"], case["dim"]
    table, lens = s["table"].long(), s["lens"].long()
    kp, vp, ks, vs = s["pool"]
    T = table.shape[1] * case["page"]
    at = table.clamp(min=0)

    def values(codes, scales):
        x = codes.view(torch.uint8)[at].view(FP8).float() * scales[at][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, G, T, D)

    q = s["q"].float().view(B, L, G, H // G, D).permute(0, 2, 1, 3, 4).reshape(B, G, L * (H // G), D)
    scores = (q @ values(kp, ks).transpose(-1, -2)).view(B, G, L, H // G, T) / math.sqrt(D)
    key = torch.arange(T, device="cuda")
    pos = lens[:, None] - L + torch.arange(L, device="cuda")
    see = visible(pos[..., None], key, case)[:, None, :, None]
    weights, lse = softmax_parts(scores, see)
    v = torch.where((key < lens[:, None])[:, None, :, None], values(vp, vs), 0.0)
    out = weights.view(B, G, L * (H // G), T) @ v
    out = out.view(B, G, L, H // G, D).permute(0, 2, 1, 3, 4).reshape(B, L, H, D)
    return out.to(s["q"].dtype), lse.permute(0, 2, 1, 3).reshape(B, L, H)


def plain_window(s, case):
    B, S, H, G, D = case["B"], case["S"], case["heads"], case["kv_heads"], case["dim"]
    W, sinks = min(case["window"], S), min(case["sinks"], S)
    C = min(256, S)  # queries of a block: each block reads the keys of its band and the sinks
    n = -(-S // C)
    lens = s["lens"].long()
    pos = torch.arange(n * C, device="cuda").view(n, C)
    key = pos[:, :1] - W + 1 + torch.arange(W - 1 + C, device="cuda")
    key = torch.cat([torch.arange(sinks, device="cuda").expand(n, sinks), key], 1)
    in_band = torch.arange(key.shape[1], device="cuda") >= sinks
    p, j = pos[..., None], key[:, None]
    see = (j >= 0) & (j <= p) & torch.where(in_band, (j > p - W), (j <= p - W))
    see = see[None] & (j < lens[:, None, None, None]) & (p < lens[:, None, None, None])
    at = key.clamp(0, S - 1)
    q = torch.nn.functional.pad(s["q"].float(), (0, 0, 0, 0, 0, n * C - S))
    q = q.view(B, n, C, G, H // G, D).permute(0, 1, 3, 4, 2, 5)
    k = s["k"].float()[:, at].permute(0, 1, 3, 4, 2)[:, :, :, None]
    v = s["v"].float()[:, at].permute(0, 1, 3, 2, 4)[:, :, :, None]
    weights, lse = softmax_parts((q @ k).div_(math.sqrt(D)), see[:, :, None, None])
    out = (weights @ v).permute(0, 1, 4, 2, 3, 5).reshape(B, n * C, H, D)[:, :S]
    return out.to(s["q"].dtype), lse.permute(0, 1, 4, 2, 3).reshape(B, n * C, H)[:, :S].contiguous()


def plain_fork(s, case):
    table, lens, refs = state_of(s)
    page, pools = case["page"], s["pool"]
    src, dst = s["src"].long(), s["dst"].long()
    slot = torch.arange(table.shape[1], device="cuda")
    n = lens[src][:, None]
    rows = table[src].long()
    full = slot < n // page
    fresh = (slot * page < n) & ~(full if case["share"] else torch.zeros_like(full))
    free = (refs == 0).nonzero()[:, 0]
    pages = free[: int(fresh.sum())]
    child = torch.where(slot * page < n, rows, -1)
    if case["share"]:
        refs.index_add_(0, rows[full], torch.ones_like(rows[full], dtype=torch.int32))
    child[fresh] = pages
    refs[pages] = 1
    table[dst] = child.to(torch.int32)
    lens[dst] = lens[src]
    for t in pools:
        u = t.view(torch.uint8) if t.dtype == FP8 else t
        u[pages] = u[rows[fresh]]
    # room for the next tokens, by rows
    have = (table >= 0).sum(1, keepdim=True)
    want = -(-(lens + s["new"])[:, None] // page)
    more = (slot >= have) & (slot < want)
    pages = (refs == 0).nonzero()[: int(more.sum()), 0]
    table[more] = pages.to(torch.int32)
    refs[pages] = 1
    return pools, table, lens, refs, torch.zeros_like(s["src"]), torch.zeros_like(s["new"])


def plain_compact(s, case):
    table, lens, refs = state_of(s)
    gone = s["gone"].long()
    left = table[gone]
    refs.index_add_(0, left[left >= 0].long(), -torch.ones_like(left[left >= 0]))
    table[gone] = -1
    lens[gone] = 0
    n_used = int((refs > 0).sum())
    ids = torch.arange(refs.numel(), device="cuda")
    holes = ((refs == 0) & (ids < n_used)).nonzero()[:, 0]
    movers = ((refs > 0) & (ids >= n_used)).nonzero()[:, 0]
    moved = torch.where(refs > 0, ids, -1)
    moved[movers] = holes
    for t in s["pool"]:
        u = t.view(torch.uint8) if t.dtype == FP8 else t
        u[holes] = u[movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    table.copy_(torch.where(table >= 0, moved[table.clamp(min=0).long()], -1))
    return (s["pool"], table, lens, refs, torch.tensor([n_used], dtype=torch.int32, device="cuda"),
            moved.to(torch.int32))


# ---- the work that a pass cannot do without


def pairs(pos0, count, case):
    """Visible keys of the queries at pos0 .. pos0 + count - 1, summed."""
    total = 0
    for p in range(pos0, pos0 + count):
        if p < 0:
            continue
        w = case["window"]
        total += p + 1 if not w or p + 1 <= w else w + min(case["sinks"], p + 1 - w)
    return total


def work(case):
    op, D = case["op"], case["dim"]
    if op == "append":
        held, new = lengths(case)
        row = case["kv_heads"] * D
        return {"bytes": 2 * sum(new) * row * 3 + 2 * 4 * case["kv_heads"] * sum(-(-n // case["page"]) for n in new),
                "flops": 0}
    if op == "attend":
        L, H, G = case["L"], case["heads"], case["kv_heads"]
        tokens = flops = 0
        for n in lengths(case):
            read = n
            if case["window"]:
                read = min(n, case["window"] + L - 1 + case["sinks"])
            tokens += read
            flops += 4 * D * H * pairs(n - L, L, case)
        return {"bytes": 2 * tokens * G * D + 8 * tokens * G // case["page"] + case["B"] * L * H * (4 * D + 4),
                "flops": flops}
    if op == "window":
        total = sum(lengths(case))
        flops = 4 * D * case["heads"] * sum(pairs(0, n, case) for n in lengths(case))
        rows = case["B"] * case["S"]
        return {"bytes": total * (2 * case["heads"] + 4 * case["kv_heads"]) * D + rows * case["heads"] * (2 * D + 4),
                "flops": flops}
    size = 2 * case["kv_heads"] * (case["page"] * D + 4)
    lens, page = lengths(case), case["page"]
    held = [-(-n // page) for n in lens]
    if op == "fork":
        copied = sum((1 if n % page else 0) if case["share"] else h for n, h in zip(lens, held)) * case["forks"]
        return {"bytes": 2 * copied * size + 4 * (1 + case["forks"]) * sum(held), "flops": 0}
    # about half of the sequences stay, and half of their pages lie behind the new end
    return {"bytes": 2 * size * sum(held) / 4 + 8 * sum(held), "flops": 0}


# ---- the same in 64 bits, from the definitions


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # pages move as they are: nothing is computed
    s = prepare(case, seed)
    return {"append": exact_append, "attend": exact_attend, "window": exact_window}[case["op"]](s, case)


def exact_append(s, case):
    """Sequence by sequence and page by page."""
    page = case["page"]
    if sum(lengths(case)[1]) // page + case["B"] > 4000:
        return None
    pools = [s["pool"][0].double(), s["pool"][1].double(), s["pool"][2].double(), s["pool"][3].double()]
    table, lens, new = s["table"].tolist(), s["lens"].tolist(), s["new"].tolist()
    for b in range(case["B"]):
        done = 0
        while done < new[b]:
            at = lens[b] + done
            p, off = table[b][at // page], at % page
            n = min(page - off, new[b] - done)
            for codes, scales, rows in ((pools[0], pools[2], s["k"]), (pools[1], pools[3], s["v"])):
                x = rows[b, done: done + n].double().transpose(0, 1)
                amax = x.abs().amax((1, 2))
                scale = torch.exp2(torch.round(torch.log2(amax.clamp(min=1e-300) / 448)))  # one of two neighbours
                scale = torch.where(448 * scale < amax, 2 * scale, scale)
                scale = torch.where(amax > 0, scale, 0.0)
                if off:
                    old = scales[p].clone()
                    scale = torch.maximum(scale, old)
                    codes[p, :, :off] = on_grid(codes[p, :, :off] * (old / scale)[:, None, None])
                codes[p, :, off: off + n] = on_grid(x / scale[:, None, None])
                scales[p] = scale
            done += n
    return pools


def on_grid(x):
    """The e4m3 value nearest to x, ties to the even one."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -9))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact_rows(q, k, v, see):
    """One sequence: q [n, H, D], k and v [t, G, D], see [n, t], in 64 bits."""
    n, H, D = q.shape
    G = k.shape[1]
    q = q.double().reshape(n, G, H // G, D)
    scores = torch.einsum("ngrd,tgd->ngrt", q, k) / D ** 0.5
    scores = torch.where(see[:, None, None], scores, -math.inf)
    lse = torch.logsumexp(scores, -1)
    weights = torch.exp(scores - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    return torch.einsum("ngrt,tgd->ngrd", weights, v).reshape(n, H, D), lse.reshape(n, H)


def exact_attend(s, case):
    if case["B"] * case["tokens"] * case["kv_heads"] > 1 << 23:
        return None
    out, lse = [], []
    kp, vp, ks, vs = s["pool"]
    for b, n in enumerate(s["lens"].tolist()):
        ids = s["table"][b, : -(-n // case["page"])].long()

        def tokens(codes, scales):
            x = codes.view(torch.uint8)[ids].view(FP8).double() * scales[ids].double()[..., None, None]
            return x.transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])[:n]

        pos = n - case["L"] + torch.arange(case["L"], device="cuda")
        key = torch.arange(n, device="cuda")
        o, l = exact_rows(s["q"][b], tokens(kp, ks), tokens(vp, vs), visible(pos[:, None], key, case))
        out.append(o)
        lse.append(l)
    return torch.stack(out), torch.stack(lse)


def exact_window(s, case):
    """Query block by query block over all the keys that any of its queries may see."""
    if case["B"] * case["S"] * case["heads"] * min(case["S"], case["window"] + 512) > 1 << 31:
        return None
    B, S, H, D = case["B"], case["S"], case["heads"], case["dim"]
    out = torch.zeros((B, S, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, S, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        for lo in range(0, n, 256):
            hi = min(n, lo + 256)
            first = max(0, lo - case["window"] + 1)
            key = torch.arange(first, hi, device="cuda")
            key = torch.cat([torch.arange(min(case["sinks"], first), device="cuda"), key])
            see = visible(torch.arange(lo, hi, device="cuda")[:, None], key, case)
            k, v = s["k"][b, key].double(), s["v"][b, key].double()
            out[b, lo:hi], lse[b, lo:hi] = exact_rows(s["q"][b, lo:hi], k, v, see)
    return out, lse
