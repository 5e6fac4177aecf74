"""Plain 64-bit forms of the K/V-cache and window attention calls (CPU
tensors), and how far the kernels may be from them.

Tolerances, from the arithmetic.  Scores: fp32 sums of D products, and in the
cache attention the query as two or three e4m3 terms whose absolute floor is
2^-18 of the row's largest magnitude: |ds| <= 2^-16 * T with T = scale *
max|q| * sum|k|, the largest over the visible keys.  Weights: rounded before
the value product with a relative error of at most `step` (half a step of the
type: 2^-8 bf16, 2^-11 fp16; two e4m3 terms: 2^-4 * 2^-4), so the
numerator moves by at most (step + 2 |ds|) * W with W the weighted mean of |v|;
below 2^-18 of the largest weight an absolute floor of 2^-19 of it applies to
each of the n tokens, n * 2^-19 * max|v| / sum of weights, where the sum is at
least the largest weight, 1.  The output is rounded once (half a step of its type); lse
moves by |ds| plus a few units of fp32."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def visible(pos, key, window, n_sink):
    see = (key <= pos) & (key >= 0)
    if window:
        see &= (key > pos - window) | (key < n_sink)
    return see


def attend(q, k, v, see, scale):
    """q [n, H, D], k and v [t, G, D], see [n, t]: (out, lse, W, T) in 64 bits."""
    n, H, D = q.shape
    t, G = k.shape[:2]
    out = torch.zeros(n, H, D, dtype=torch.float64)
    wabs = torch.zeros(n, H, D, dtype=torch.float64)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64)
    top = torch.zeros(n, H, dtype=torch.float64)
    for i in range(n):
        idx = see[i].nonzero()[:, 0]
        if not len(idx):
            continue
        for h in range(H):
            kk, vv = k[idx, h // (H // G)].double(), v[idx, h // (H // G)].double()
            s = scale * (kk @ q[i, h].double())
            lse[i, h] = torch.logsumexp(s, 0)
            w = torch.exp(s - lse[i, h])
            out[i, h] = w @ vv
            wabs[i, h] = w @ vv.abs()
            top[i, h] = scale * q[i, h].double().abs().max() * kk.abs().sum(1).max()
    return out, lse, wabs, top


def dequantise(codes, scale):
    """[n_pages, H, page, D] codes and [n_pages, H] scales -> fp64 values."""
    return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None, None]


def cache_tokens(kp, ks, table_row, n, page):
    """(values [n, H, D] with zeros for missing pages, there [n]) of one sequence."""
    n_pages, H, _, D = kp.shape
    out = torch.zeros(max(n, 0), H, D, dtype=torch.float64)
    there = torch.zeros(max(n, 0), dtype=torch.bool)
    for j in range(0, max(n, 0), page):
        p = int(table_row[j // page])
        if 0 <= p < n_pages:
            m = min(page, n - j)
            out[j: j + m] = dequantise(kp[p: p + 1], ks[p: p + 1])[0].transpose(0, 1)[:m]
            there[j: j + m] = True
    return out, there


def cache_attention(q, kp, vp, ks, vs, table, lens, window=0, n_sink=0, scale=0.0):
    B, L, H, D = q.shape
    page = kp.shape[2]
    scale = scale or D ** -0.5
    parts = []
    for b in range(B):
        n = min(int(lens[b]), table.shape[1] * page)
        k, there = cache_tokens(kp, ks, table[b], n, page)
        v, _ = cache_tokens(vp, vs, table[b], n, page)
        pos = int(lens[b]) - L + torch.arange(L)
        see = visible(pos[:, None], torch.arange(max(n, 0)), window, n_sink) & there
        parts.append(attend(q[b], k, v, see, scale))
    return [torch.stack(x) for x in zip(*parts)]


def window_attention(q, k, v, window, n_sink=0, lens=None, scale=0.0):
    B, S, H, D = q.shape
    scale = scale or D ** -0.5
    parts = []
    for b in range(B):
        n = S if lens is None else min(max(int(lens[b]), 0), S)
        pos = torch.arange(S)[:, None]
        see = visible(pos, torch.arange(n), window, n_sink) & (pos < n)
        parts.append(attend(q[b], k[b], v[b], see, scale))
    return [torch.stack(x) for x in zip(*parts)]


def check(got, want, step, vmax, n_keys):
    """got = (out, lse) of a kernel (any device) against attend()'s four."""
    out, lse = got[0].cpu(), got[1].cpu().double()
    ref, rlse, wabs, top = want
    half = HALF_STEP[out.dtype]
    ds = 2.0 ** -16 * top
    err = (out.double() - ref).abs()
    tiny = torch.finfo(out.dtype).tiny * torch.finfo(out.dtype).eps
    tol = (step + 2 * ds[..., None]) * wabs + n_keys * 2.0 ** -19 * vmax + half * ref.abs() * (1 + step) + tiny
    assert torch.isfinite(out).all()
    worst = (err - tol).max().item()
    assert worst <= 0, f"out off by {err.max().item():.3g}, {worst:.3g} over the tolerance"
    empty = torch.isneginf(rlse)
    assert torch.equal(empty, torch.isneginf(lse)), "other rows are empty"
    assert (out[empty] == 0).all()
    d = (lse[~empty] - rlse[~empty]).abs() - ds[~empty] - 2.0 ** -20 * (1 + rlse[~empty].abs())
    assert not d.numel() or d.max().item() <= 0, f"lse {d.max().item():.3g} over the tolerance"


# ---- the cache's own calls, on a state of Python integers


def power_scale(amax):
    """The least power of two s with amax <= 448 s."""
    if amax == 0:
        return 0.0
    s = 2.0 ** (math.floor(math.log2(amax)) - 9)
    while 448 * s < amax:
        s *= 2
    return max(s, 2.0 ** -126)


def append(kp, ks, k, table, lens, n_new):
    """One of K or V: returns new (codes uint8, scales) after the rows k [B, L, H, D]."""
    codes, scales = kp.view(torch.uint8).clone(), ks.clone()
    n_pages, H, page, D = kp.shape
    B, L = k.shape[:2]
    for b in range(B):
        n0, nn = int(lens[b]), min(max(int(n_new[b]), 0), L)
        pages = {}
        for i in range(nn):
            at = n0 + i
            if at >= 0 and at // page < table.shape[1]:
                pages.setdefault(at // page, []).append(i)
        for j, rows in pages.items():
            p = int(table[b, j])
            if not 0 <= p < n_pages:
                continue
            off = (n0 + rows[0]) % page
            for h in range(H):
                x = k[b, rows, h].float()
                finite = x[torch.isfinite(x)].abs()
                s = power_scale(finite.max().item() if finite.numel() else 0.0)
                old = scales[p, h].item() if off else 0.0
                new = max(s, old)
                if off and new > old:
                    value = codes[p, h, :off].view(torch.float8_e4m3fn).float() * old
                    codes[p, h, :off] = (value / new).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                y = x / new if new > 0 else x
                codes[p, h, off: off + len(rows)] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                scales[p, h] = new
    return codes, scales


def leading(row, n_pages):
    out = []
    for p in row:
        if not 0 <= p < n_pages:
            break
        out.append(p)
    return out


def reserve(table, lens, refs, n_new, page):
    """Lists in, (table, refs, status) out."""
    table, refs = [list(r) for r in table], list(refs)
    n_pages, width = len(refs), len(table[0])
    free = [p for p in range(n_pages) if refs[p] <= 0]
    run, status = 0, []
    for b, row in enumerate(table):
        have = len(leading(row, n_pages))
        want = -(-max(lens[b] + n_new[b], 0) // page) if n_new[b] > 0 else 0
        if want > width:
            status.append(2)
            continue
        need = max(want - have, 0)
        if need and run + need > len(free):
            run += need
            status.append(1)
            continue
        for j in range(need):
            row[have + j] = free[run + j]
            refs[free[run + j]] = 1
        run += need
        status.append(0)
    return table, refs, status


def fork(table, lens, refs, src, dst, page, share):
    """Lists in, (table, lens, refs, status, copies) out; copies are (from, to) pages."""
    before, lens0 = [list(r) for r in table], list(lens)
    table, lens, refs = [list(r) for r in table], list(lens), list(refs)
    n_pages, width, n_seq = len(refs), len(table[0]), len(table)
    free = [p for p in range(n_pages) if refs[p] <= 0]
    run, status, copies, named = 0, [], [], set()
    for s, d in zip(src, dst):
        again = d in named
        named.add(d)
        if not (0 <= s < n_seq and 0 <= d < n_seq) or lens0[d] != 0 or leading(before[d], n_pages) or again:
            status.append(2)
            continue
        n = max(lens0[s], 0)
        pages = leading(before[s], n_pages)[: -(-n // page)]
        n = min(n, len(pages) * page)
        full = n // page if share else 0
        need = len(pages) - full
        if need and run + need > len(free):
            run += need
            status.append(1)
            continue
        new = free[run: run + need]
        for p in pages[:full]:
            refs[p] += 1
        for a, p in zip(pages[full:], new):
            copies.append((a, p))
            refs[p] = 1
        run += need
        table[d] = (pages[:full] + new + [-1] * width)[:width]
        lens[d] = n
        status.append(0)
    return table, lens, refs, status, copies


def free(table, lens, refs, rows):
    table, lens, refs = [list(r) for r in table], list(lens), list(refs)
    for r in rows:
        if 0 <= r < len(table):
            for p in table[r]:
                if 0 <= p < len(refs):
                    refs[p] -= 1
            table[r] = [-1] * len(table[r])
            lens[r] = 0
    return table, lens, refs


def compact(table, refs):
    """(table, refs, used, moved, copies)."""
    table, refs = [list(r) for r in table], list(refs)
    n = len(refs)
    used = sum(r > 0 for r in refs)
    holes = [p for p in range(used) if refs[p] <= 0]
    movers = [p for p in range(used, n) if refs[p] > 0]
    moved = [p if refs[p] > 0 else -1 for p in range(n)]
    for a, b in zip(movers, holes):
        moved[a] = b
        refs[b], refs[a] = refs[a], 0
    table = [[moved[p] if used <= p < n else p for p in row] for row in table]
    return table, refs, used, moved, list(zip(movers, holes))
