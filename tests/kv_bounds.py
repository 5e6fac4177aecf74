"""Sharper bounds for the attention calls than a tolerance that is one number:
per output, from the weights and values that it is made of.

With e_j = exp(s_j - max s), Z = sum e_j >= 1 and w_j = e_j / Z over the keys
that a row sees, out = sum_j w_j v_j.  The error of one weight moves the output
by at most

    amp_j = (step + 2 ds) w_j |v_j| + floor M / Z |v_j| / vs_j

- step: the rounding of a weight relative to itself.  Window: half a step of
  the inputs' type.  Cache: the weight is rounded to half precision (2^-11), then
  to the sum of two e4m3 terms (2^-4 * 2^-4; bf16) or three (2^-12; fp16).
- floor: the same where the last term has left its normal numbers.  Window: fp16
  weights are taken relative to a reference that is at most twice the largest
  one, half a subnormal step is 2^-25.  Cache: a weight times its page's value
  scale vs is stored times 256 / (a reference of at most 2 M), M the largest such
  product, and term i times 2^(4 i): half a subnormal step of e4m3 (2^-10) is
  2^-14 under two terms, 2^-18 under three, of 256 / 2.
- ds: the scores' error, 2^-16 scale max|q| sum|k| (fp32 sums; the query's terms).

Beside them: fp32 sums (2^-20 of sum w|v|) and one rounding of the output.  All
of them together bound every single output (tol).  They are independent
roundings of many weights, whose squares add up: over many outputs the mean of
(error / unit)^2, unit^2 the sum of the squares, is below 1 (a uniform rounding
error has a third of its bound's square), and that is what a lost part of a long
sum cannot hide from."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
WINDOW = {torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -24)}
CACHE = {torch.bfloat16: (2.0 ** -8 + 2.0 ** -11, 2.0 ** -21), torch.float16: (2.0 ** -11 + 2.0 ** -12, 2.0 ** -25)}


def attend(q, k, v, see, scale, step, floor, half, vs=None):
    """q [n, H, D], k and v [t, G, D], see [n, t], vs [t, G]: (out, lse, tol, unit, dlse) in 64 bits."""
    n, H, D = q.shape
    t, G = k.shape[:2]
    out, tol, unit = [torch.zeros(n, H, D, dtype=torch.float64) for _ in range(3)]
    lse = torch.full((n, H), -math.inf, dtype=torch.float64)
    dlse = torch.zeros(n, H, dtype=torch.float64)
    q, k, v = q.double(), k.double(), v.double()
    for i in range(n):
        idx = see[i].nonzero()[:, 0]
        if not len(idx):
            continue
        for g in range(G):
            hs = slice(g * (H // G), (g + 1) * (H // G))
            kk, vv, qq = k[idx, g], v[idx, g], q[i, hs]
            s = scale * (qq @ kk.T)
            top = s.amax(1, keepdim=True)
            e = torch.exp(s - top)
            Z = e.sum(1, keepdim=True)
            w = e / Z
            ds = 2.0 ** -16 * scale * qq.abs().amax(1) * kk.abs().sum(1).amax()
            size = torch.ones(len(idx), dtype=torch.float64) if vs is None else vs[idx, g].double()
            per = torch.where(size > 0, 1 / size, 0.0)[:, None] * vv.abs()  # a value in units of its scale
            M = (e * size).amax(1, keepdim=True)
            o, wabs = w @ vv, w @ vv.abs()
            rel = (step + 2 * ds)[:, None]
            out[i, hs] = o
            lse[i, hs] = (top + torch.log(Z))[:, 0]
            dlse[i, hs] = ds + 2.0 ** -20 * (1 + lse[i, hs].abs())
            rest = 2.0 ** -20 * wabs
            tol[i, hs] = rel * wabs + floor * M / Z * per.sum(0) + rest + half * o.abs() * (1 + step)
            unit[i, hs] = torch.sqrt(rel ** 2 * (w ** 2 @ vv ** 2) + (floor * M / Z) ** 2 * (per ** 2).sum(0) +
                                     rest ** 2 + (half * o) ** 2)
    return out, lse, tol, unit, dlse


def visible(pos, key, window, n_sink):
    see = (key <= pos) & (key >= 0)
    if window:
        see &= (key > pos - window) | (key < n_sink)
    return see


def cache_attention(q, kp, vp, ks, vs, table, lens, window=0, n_sink=0, scale=0.0):
    """Codes [n_pages, G, page, D] (uint8) and scales [n_pages, G] of a cache, all on the CPU."""
    B, L, H, D = q.shape
    n_pages, G, page, _ = kp.shape
    scale = scale or D ** -0.5
    step, floor = CACHE[q.dtype]
    parts = []
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        ids = table[b, : -(-n // page)].long()
        there = ((ids >= 0) & (ids < n_pages)).repeat_interleave(page)[:n]
        at = ids.clamp(0, n_pages - 1)

        def tokens(codes, sc):
            x = codes[at].view(torch.float8_e4m3fn).double() * sc[at].double()[..., None, None]
            return x.transpose(1, 2).reshape(-1, G, D)[:n]

        pos = n - L + torch.arange(L)
        see = visible(pos[:, None], torch.arange(n), window, n_sink) & there
        parts.append(attend(q[b], tokens(kp, ks), tokens(vp, vs), see, scale, step, floor, HALF_STEP[q.dtype],
                            vs[at].double().repeat_interleave(page, 0)[:n]))
    return [torch.stack(x) for x in zip(*parts)]


def window_attention(q, k, v, window, n_sink=0, lens=None, scale=0.0):
    B, S, H, D = q.shape
    scale = scale or D ** -0.5
    step, floor = WINDOW[q.dtype]
    parts = []
    for b in range(B):
        n = S if lens is None else min(max(int(lens[b]), 0), S)
        pos = torch.arange(S)[:, None]
        see = visible(pos, torch.arange(n), window, n_sink) & (pos < n)
        kk, vv = k[b].clone(), v[b].clone()
        kk[n:], vv[n:] = 0, 0  # (padding may hold anything)
        parts.append(attend(q[b].nan_to_num(0.0), kk, vv, see, scale, step, floor, HALF_STEP[q.dtype]))
    return [torch.stack(x) for x in zip(*parts)]


def check(out, lse, want, sharp=2.0 ** -4):
    """out and lse of a kernel (any device) against the five above; `sharp`: what the bound has to be below,
    relative to the outputs' own size, for the check to mean something (at the median)."""
    ref, rlse, tol, unit, dlse = want
    tiny = torch.finfo(out.dtype).tiny * torch.finfo(out.dtype).eps
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(out).all(), "not finite"
    empty = torch.isneginf(rlse)
    assert torch.equal(empty, torch.isneginf(lse)), "other rows are empty"
    assert (out[empty] == 0).all(), "an empty row is not zero"
    if empty.all():
        return
    err = (out - ref).abs()[~empty]
    tol, unit, size = tol[~empty] + tiny, unit[~empty] + tiny, ref[~empty].abs()
    if sharp:
        assert (tol / size).median().item() < sharp, "the bound is too wide to show anything"
    worst = (err - tol).max().item()
    assert worst <= 0, f"out off by {err.max().item():.3g}, {worst:.3g} over its bound"
    rms = (err / unit).square().mean().sqrt().item()
    assert rms <= 1, f"out: {rms:.3g} times the bound on average"
    d = (lse - rlse).abs()[~empty] - dlse[~empty]
    assert d.max().item() <= 0, f"lse {d.max().item():.3g} over its bound"
