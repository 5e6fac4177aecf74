"""Edges of the K/V-cache and window attention calls on a GPU: values that are
not finite, scales and lengths out of the ordinary, waits that run out, other
streams."""
import pytest
import torch

from tests.test_gpu_cache import _cuda, _gen, _i32, _run_append

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("rows", [1, 3, -1, "a page and 3"])
def test_append_scale_beside_values_that_are_not_finite(dtype, D, page, rows):
    """A sequence for each place of an infinity or NaN in 8 neighbours and each
    place of the largest finite value among the others: the scale is that
    value's, in one row, a few, all but one of a page, a page and a few."""
    L = page + 3 if isinstance(rows, str) else rows if rows > 0 else page - 1
    pairs = [(i, j) for i in range(8) for j in range(8) if i != j]
    B, H, per = len(pairs), 2, -(-L // page)
    g = _gen(D + page + L)
    x = [torch.full((B, L, H, D), 0.01), torch.full((B, L, H, D), -0.02)]
    for b, (i, j) in enumerate(pairs):
        for h in range(H):
            for t, bad in zip(x, ("inf", "nan") if b % 2 else ("nan", "-inf")):
                row = L - 1 if b % 3 == 0 else int(torch.randint(0, L, (1,), generator=g))
                at = 8 * int(torch.randint(0, D // 8, (1,), generator=g))
                t[b, row, h, at + i] = float(bad)
                t[b, row, h, at + j] = 100.0
    pool = [torch.zeros((B * per, H, page, D), dtype=torch.uint8) for _ in range(2)] + [
        torch.zeros((B * per, H)) for _ in range(2)]
    table = torch.arange(B * per, dtype=torch.int32).view(B, per)
    _run_append(pool, x[0].to(dtype), x[1].to(dtype), table, torch.zeros(B, dtype=torch.int32), None)


@pytest.mark.parametrize("page", [16, 64, 128])
def test_append_step_that_is_not_finite(page):
    """A decode step into a page that is partly full: the row's finite values decide about the growth of the scale."""
    g = _gen(page)
    B, H, D = 8, 2, 128
    pool = [torch.randint(0, 0x70, (B, H, page, D), generator=g, dtype=torch.int16).to(torch.uint8) for _ in range(2)]
    pool += [torch.full((B, H), 2.0 ** -8) for _ in range(2)]
    k = torch.randn((B, 1, H, D), generator=g)
    for b in range(B):
        k[b, 0, 0, 40] = float("inf")
        k[b, 0, 1, 8 * b] = float("nan")
        k[b, 0, :, 41 + b] = 50.0 * 2.0 ** b
    _run_append(pool, k.bfloat16(), -k.half().bfloat16(), torch.arange(B, dtype=torch.int32)[:, None],
                _i32([page - 1 - b for b in range(B)]), None)
