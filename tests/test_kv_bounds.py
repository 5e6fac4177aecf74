"""The bounds of tests/kv_bounds.py reject wrong outputs: the kernels' own
arithmetic, emulated, passes; planted mistakes do not."""
import pytest
import torch

from tests import kv_bounds


def cache(n, page, G, D, seed, dtype, H):
    """A sequence of n tokens with positive values, some pages much larger than others."""
    g = torch.Generator()
    g.manual_seed(seed)
    n_pages = -(-n // page)
    kp = torch.randint(0, 256, (n_pages, G, page, D), generator=g, dtype=torch.int16)
    kp = torch.where(kp % 128 > 0x50, kp - 0x38, kp).to(torch.uint8)
    vp = torch.randint(0x30, 0x71, (n_pages, G, page, D), generator=g, dtype=torch.int16).to(torch.uint8)
    ks = torch.full((n_pages, G), 2.0 ** -4)
    vs = torch.exp2(torch.randint(-9, -5, (n_pages, G), generator=g).float()) * (1 + torch.rand((n_pages, G), generator=g))
    vs[torch.randperm(n_pages, generator=g)[: -(-n_pages // 20)]] *= 16
    table = torch.randperm(n_pages, generator=g).int()[None]
    q = (torch.randn((1, 1, H, D), generator=g) * 0.5).to(dtype)
    return q, kp, vp, ks, vs, table, torch.tensor([n], dtype=torch.int32)


def emulate(q, kp, vp, ks, vs, table, lens, terms, drop=None):
    """The cache kernel's arithmetic with `terms` e4m3 terms a weight, tile by tile, in 64 bits elsewhere."""
    H, D = q.shape[2:]
    G, page = kp.shape[1:3]
    n = int(lens[0])
    ids = table[0].long()
    out, lse = [], []
    for h in range(H):
        g = h // (H // G)
        k = (kp[ids, g].view(torch.float8_e4m3fn).double() * ks[ids, g].double()[:, None, None]).reshape(-1, D)[:n]
        code = vp[ids, g].view(torch.float8_e4m3fn).double().reshape(-1, D)[:n]
        size = vs[ids, g].double().repeat_interleave(page)[:n]
        s = D ** -0.5 * (k @ q[0, 0, h].double())
        e = torch.exp(s - s.max())
        acc = torch.zeros(D, dtype=torch.float64)
        for t in range(0, n, 128):
            if drop is not None and drop[0] <= t < drop[1]:
                continue
            product = e[t: t + 128] * size[t: t + 128]
            unit = product.max() * 1.3 / 256  # a reference between 1 and 2 times the largest
            x = (product / unit).half()
            for i in range(terms):
                c = x.to(torch.float8_e4m3fn).half()
                acc += (c.double() @ code[t: t + 128]) * unit * 2.0 ** (-4 * i)
                x = (x - c) * 16
        out.append(acc / e.sum())
        lse.append(torch.logsumexp(s, 0))
    return torch.stack(out)[None, None].to(q.dtype), torch.stack(lse)[None, None]


TERMS = {torch.bfloat16: 2, torch.float16: 3}
SIZES = [(3, 16), (200, 16), (6000, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,page", SIZES)
def test_the_kernels_arithmetic_passes(dtype, n, page):
    x = cache(n, page, 2, 64, n, dtype, 8)
    kv_bounds.check(*emulate(*x, TERMS[dtype]), kv_bounds.cache_attention(*x))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_mistakes_do_not_pass(dtype):
    n, page = 6000, 64
    x = cache(n, page, 2, 64, 1, dtype, 8)
    want = kv_bounds.cache_attention(*x)
    out, lse = emulate(*x, TERMS[dtype])
    wrong = {"zeros": torch.zeros_like(out), "heads swapped": out.flip(2),
             "a hundredth too large": (out.double() * 1.01).to(dtype),
             "a split lost": emulate(*x, TERMS[dtype], drop=(2560, 2944))[0]}
    vs = x[4].clone()
    vs[int(x[5][0, 40])] *= 2
    wrong["a page under another scale"] = emulate(*x[:4], vs, *x[5:], TERMS[dtype])[0]
    for o in wrong.values():
        with pytest.raises(AssertionError):
            kv_bounds.check(o, lse, want)
    with pytest.raises(AssertionError):
        kv_bounds.check(out, lse + 1e-3, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [2, 3, 5])
def test_a_lost_term_does_not_pass(dtype, n):
    """Of few tokens, whose weights' roundings do not average out."""
    x = cache(n, 16, 4, 128, n + 10, dtype, 64)
    want = kv_bounds.cache_attention(*x)
    kv_bounds.check(*emulate(*x, TERMS[dtype]), want)
    with pytest.raises(AssertionError):
        kv_bounds.check(*emulate(*x, TERMS[dtype] - 1), want)
