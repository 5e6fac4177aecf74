"""Edges of the K/V-cache and window attention calls on a GPU: values that are
not finite, scales and lengths out of the ordinary, waits that run out, other
streams.  Outputs of the attentions are held to the bounds of tests/kv_bounds.py."""
import pytest
import torch

from tests import kv_bounds
from tests.test_gpu_cache import _cuda, _gen, _i32, _run_append

pytestmark = pytest.mark.gpu

import streaming_top_b200 as si  # noqa: E402


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


# ------------------------------------------------------------------ attention over the cache


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [0.0, 1e-10, 1e-38])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (30, 3)])
def test_cache_attention_of_queries_that_are_zero(dtype, scale, window, n_sink):
    """Queries of zeros, or nearly, at any score scale: the mean of what they see, ln of its count."""
    g = _gen(50)
    page, D, lens = 16, 64, [200, 77]
    kp, vp = [torch.randint(0x30, 0x71, (30, 1, page, D), generator=g, dtype=torch.int16).to(torch.uint8) for _ in range(2)]
    ks = vs = torch.full((30, 1), 2.0 ** -7)
    table = torch.randperm(30, generator=g).int().view(2, 15)
    q = torch.zeros((2, 2, 8, D), dtype=dtype)
    q[:, :, 1::2] = torch.finfo(dtype).tiny if scale else 0
    out, lse = si.cache_attention(q.cuda(), si.PagedCache(*_cuda(kp, vp, ks, vs)), table.cuda(), _i32(lens).cuda(),
                                  scale=scale, window=window, n_sink=n_sink)
    for b, n in enumerate(lens):
        v = vp[table[b].long()].view(torch.float8_e4m3fn).double().reshape(-1, D) * 2.0 ** -7
        for i in range(2):
            p = n - 2 + i
            see = [j for j in range(p + 1) if not window or j > p - window or j < n_sink]
            # a weight (equal ones: 256, exact in every form) and fp32 sums, then one rounding of the output
            half = torch.finfo(dtype).eps / 2
            assert torch.allclose(out[b, i].cpu().double(), v[see].mean(0).expand(8, D), rtol=half + 2.0 ** -18, atol=0)
            assert torch.allclose(lse[b, i].cpu().double(), torch.tensor(float(len(see))).double().log(), rtol=2.0 ** -20)


def _cache(pool):
    return si.PagedCache(*_cuda(*pool))


def _check_cache(q, pool, table, lens, sharp=2.0 ** -4, **kw):
    """cache_attention against the bounds; `sharp` as in kv_bounds.check."""
    word = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = si.cache_attention(q.cuda(), _cache(pool), table.cuda(), lens.cuda(), device_status=word, **kw)
    assert word.eq(0).all()
    kv_bounds.check(out, lse, kv_bounds.cache_attention(q, *pool, table, lens, **kw), sharp)
    return out, lse


def _positive(n_pages, G, page, D, g):
    """A pool with keys of every sign and positive values, whose sums do not cancel."""
    k = torch.randint(0, 256, (n_pages, G, page, D), generator=g, dtype=torch.int16)
    k = torch.where(k % 128 > 0x50, k - 0x38, k).to(torch.uint8)
    v = torch.randint(0x30, 0x71, (n_pages, G, page, D), generator=g, dtype=torch.int16).to(torch.uint8)
    return [k, v, torch.full((n_pages, G), 2.0 ** -4), torch.full((n_pages, G), 2.0 ** -7)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,H,L", [(128, 4, 1), (64, 4, 2), (128, 64, 1), (64, 64, 1), (128, 20, 1)])
@pytest.mark.parametrize("apart", [6, 10, 14, 18, 30, 60])
def test_cache_attention_weight_on_a_page_of_small_values(dtype, D, H, L, apart):
    """All the weight lies on one page whose value scale is 2^-apart of its
    neighbours': its values come out as exactly as any."""
    g = _gen(apart)
    page, n = 16, 300
    n_pages = -(-n // page)
    pool = _positive(n_pages, 1, page, D, g)
    table = torch.randperm(n_pages, generator=g).int()[None]
    for j in (2, 7, 9, 17):  # in the first tile, at its end, in the second, in the last
        k, v, ks, vs = [t.clone() for t in pool]
        k &= 0x8F  # small beside the first dim
        p = int(table[0, j])
        k[..., 0] = 0xB8  # -1
        k[p, :, :, 0] = 0x38  # 1
        vs[:] = 2.0 ** (apart - 3)
        vs[p] = 2.0 ** -3
        q = torch.randn((1, L, H, D), generator=g) * 0.1
        q[..., 0] = (0.7 * (apart + 30)) * D ** 0.5 / 2 / 2.0 ** -4  # a score difference of 0.7 (apart + 30)
        _check_cache(q.to(dtype), (k, v, ks, vs), table, _i32([n]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("H", [4, 64])
def test_cache_attention_beside_a_page_of_large_scale(dtype, window, H):
    """Pages whose scale is 2^10 of the others': their visible values are zeros
    (what made the scale large lies before the window), the others' count."""
    g = _gen(window + H)
    page, n, D = 16, 200, 128
    n_pages = -(-n // page)
    pool = _positive(n_pages, 1, page, D, g)
    table = torch.randperm(n_pages, generator=g).int()[None]
    for j in (3, (n - 70) // page):
        p = int(table[0, j])
        pool[3][p] *= 2.0 ** 10
        pool[1][p, :, (n - 70) % page if window else 0:] = 0
    q = (torch.randn((1, 1, H, D), generator=g) * 0.3).to(dtype)
    _check_cache(q, pool, table, _i32([n]), window=window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_cache_attention_weight_on_zeros(dtype):
    """A page of scale zero takes nearly all the weight; the small rest is the output, and lse counts both."""
    g = _gen(51)
    pool = _positive(10, 1, 16, 128, g)
    table = torch.arange(10, dtype=torch.int32)[None]
    pool[0] &= 0x8F
    pool[0][..., 0] = 0xB8
    pool[0][4, :, :, 0] = 0x38
    pool[3][4] = 0.0
    q = torch.randn((1, 1, 8, 128), generator=g) * 0.1
    q[..., 0] = 4.0 * 128 ** 0.5 / 2 / 2.0 ** -4  # a score difference of 4
    _check_cache(q.to(dtype), pool, table, _i32([150]))
    pool[3][:] = 0.0
    out, _ = si.cache_attention(q.to(dtype).cuda(), _cache(pool), table.cuda(), _i32([150]).cuda())
    assert (out == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,L", [(2, 1), (16, 1), (64, 1), (12, 3)])
def test_cache_attention_of_a_long_context_to_its_bounds(dtype, H, L):
    """Sequences of tens of thousands of tokens, cut between blocks and joined,
    some pages with much larger values than others: a lost part would show."""
    g = _gen(H)
    lens, page, D = [40000, 13, 4000], 64, 128
    need = [-(-n // page) for n in lens]
    pool = _positive(sum(need), 1, page, D, g)
    pool[3] = torch.exp2(torch.randint(-9, -5, (sum(need), 1), generator=g).float()) * (
        1 + torch.rand((sum(need), 1), generator=g))
    order = torch.randperm(sum(need), generator=g).int()
    pool[3][order[::20].long()] *= 16
    table = torch.full((3, max(need)), -1, dtype=torch.int32)
    for b, part in enumerate(order.split(need)):
        table[b, : need[b]] = part
    q = (torch.randn((3, L, H, D), generator=g) * 0.5).to(dtype)
    _check_cache(q, pool, table, _i32(lens))
    _check_cache(q, pool, table, _i32(lens), window=3000, n_sink=40)


@pytest.mark.parametrize("n", [1, 2, 3, 5])
def test_cache_attention_of_few_tokens_has_all_its_bits(n):
    """fp16 keeps its 11 bits, bf16 its 8: of few tokens, whose roundings do not average out."""
    for dtype in (torch.bfloat16, torch.float16):
        g = _gen(n)
        pool = _positive(40, 4, 16, 128, g)
        table = torch.arange(40, dtype=torch.int32)[:, None]
        q = (torch.randn((40, 1, 64, 128), generator=g) * 0.5).to(dtype)
        _check_cache(q, pool, table, _i32([n] * 40))


@pytest.mark.parametrize("L,window,n_sink", [(1, 10, 0), (3, 10, 2), (2, 1, 0), (1, 0, 0), (4, 40, 5)])
def test_cache_attention_length_beyond_the_table_is_the_tables(L, window, n_sink):
    """A length beyond max_pages * page is read as that: the queries are the table's last tokens."""
    g = _gen(52)
    page, width = 16, 3
    pool = _positive(12, 1, page, 64, g)
    table = torch.randperm(12, generator=g).int().view(4, width)
    q = (torch.randn((4, L, 4, 64), generator=g) * 0.5).bfloat16()
    for lens in ([48, 49, 53, 1000], [2 ** 31 - 1, 48 + L, 47, 2 ** 31 - 49]):
        _check_cache(q, pool, table, _i32(lens), window=window, n_sink=n_sink)


# ------------------------------------------------------------------ prompts


def _check_window(q, k, v, window, n_sink=0, lens=None, **kw):
    word = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = si.window_attention(*_cuda(q, k, v), window=window, n_sink=n_sink,
                                   lens=None if lens is None else lens.cuda(), device_status=word, **kw)
    assert word.eq(0).all()
    kv_bounds.check(out, lse, kv_bounds.window_attention(q, k, v, window, n_sink, lens, **kw))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,n_sink", [(128, 0), (128, 4), (200, 0), (60, 100)])
@pytest.mark.parametrize("steps", [1, 7, 30])
def test_narrow_band_whose_scores_keep_growing(dtype, D, window, n_sink, steps):
    """Scores that climb by `steps` (to the base 2) every 16 keys: the reference
    moves in most column blocks, and the weights written before follow it."""
    g = _gen(steps)
    S, H = 600, 8
    q = torch.randn((1, S, H, D), generator=g) * 0.05
    k = torch.randn((1, S, 1, D), generator=g) * 0.05
    v = torch.rand((1, S, 1, D), generator=g) + 0.1
    q[..., 0] = 4.0
    climb = steps / 16 * 0.6931 * D ** 0.5 / 4.0  # a key
    k[0, :, 0, 0] = (torch.arange(S) - S / 2) * climb
    _check_window(q.to(dtype), k.to(dtype), v.to(dtype), window, n_sink)


# ------------------------------------------------------------------ waits that run out


def _runs_out(call):
    """With a load withheld the call returns, its status word says so, and the next call is right."""
    word = torch.zeros(2, dtype=torch.int32, device="cuda")
    want = call(word)
    assert word.eq(0).all()
    si.test_withhold_loads(1)
    try:
        call(word)
        torch.cuda.synchronize()
    finally:
        si.test_withhold_loads(0)
    assert int(word[0]) == si.SI_ERR_TIMEOUT and int(word[1]) > 0
    assert si.device_status() == si.SI_OK  # (the shared record was not touched)
    word.zero_()
    for a, b in zip(call(word), want):
        assert torch.equal(a, b)
    assert word.eq(0).all()


@pytest.mark.parametrize("window,n_sink", [(128, 0), (100, 4), (300, 0), (300, 20), (500, 5)])
@pytest.mark.parametrize("D", [64, 128])
def test_window_attention_wait_that_runs_out(window, n_sink, D):
    """The narrow form, key tiles of 64 and of 128, several items a block."""
    g = _gen(60)
    q, k, v = [torch.randn((1, 8192, n, D), generator=g).bfloat16().cuda() for n in (16, 2, 2)]
    _runs_out(lambda word: si.window_attention(q, k, v, window=window, n_sink=n_sink, device_status=word))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,n,window", [(4, 6000, 0), (16, 6000, 0), (64, 6000, 0), (8, 900, 0), (64, 3000, 200)])
def test_cache_attention_wait_that_runs_out(dtype, D, H, n, window):
    """Units cut between blocks and whole ones, all numbers of rows."""
    g = _gen(61)
    page, B = 64, 40
    width = -(-n // page)
    cache = _cache(_positive(B * width, 1, page, D, g))
    table = torch.randperm(B * width, generator=g).int().view(B, width).cuda()
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = (torch.randn((B, 1, H, D), generator=g) * 0.5).to(dtype).cuda()
    _runs_out(lambda word: si.cache_attention(q, cache, table, lens, window=window, device_status=word))


def test_window_attention_key_by_key_over_a_long_prompt():
    """A block that is done again key by key keeps its other warps waiting for seconds: the limits allow for it."""
    g = _gen(62)
    S, D = 600_000, 128
    q, k, v = [torch.randn((1, S, 1, D), generator=g).bfloat16() for _ in range(3)]
    v = v.abs() + 0.1
    word = torch.zeros(2, dtype=torch.int32, device="cuda")
    qd, kd, vd = _cuda(q, k, v)
    vd[0, S - 5, 0, 3] = float("nan")
    out, lse = si.window_attention(qd, kd, vd, window=S, device_status=word)
    assert word.eq(0).all()
    assert torch.isnan(out[0, S - 5:, 0, 3]).all() and torch.isnan(out).sum() == 5
    pos = torch.tensor([S - 7, S - 250, S - 300])  # in that block, and before it
    see = torch.arange(S) <= pos[:, None]
    want = kv_bounds.attend(q[0, pos], k[0], v[0], see, D ** -0.5, *kv_bounds.WINDOW[torch.bfloat16], 2.0 ** -8)
    kv_bounds.check(out[0, pos.cuda()], lse[0, pos.cuda()], want)


# ------------------------------------------------------------------ other streams


def _attention_calls():
    """{name: (a call on a stream, its inputs, where the outputs are)}, each tensor larger than the allocator's small blocks."""
    def window():
        x = [torch.randn((1, 8192, n, 64), device="cuda").bfloat16() for n in (16, 4, 4)]
        return x, lambda s: si.window_attention(*x, window=100, stream=s)

    def cache():
        pool = [torch.zeros((512, 4, 64, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
        pool += [torch.ones((512, 4), device="cuda") for _ in range(2)]
        q = torch.randn((512, 4, 16, 64), device="cuda").half()
        table = torch.arange(512, dtype=torch.int32, device="cuda")[:, None].repeat(1, 2048).contiguous()
        lens = torch.full((512,), 60, dtype=torch.int32, device="cuda")
        x = [q, table, *pool]
        return x, lambda s: si.cache_attention(q, si.PagedCache(*pool), table, lens, stream=s)

    def top_k():
        x = [torch.randn(shape, device="cuda").to(dt) for shape, dt in (
            ((1, 4096, 64, 128), torch.bfloat16), ((1, 8192, 128), torch.bfloat16), ((1, 4096, 64), torch.float32))]
        return x, lambda s: si.indexer_topk(*x, 4, 128, stream=s)

    def sparse():
        q = torch.randn((1, 256, 64, 576), device="cuda").bfloat16()
        kv = torch.randn((1, 1024, 576), device="cuda").bfloat16()
        idx = torch.randint(0, 1024, (1, 256, 128), dtype=torch.int32, device="cuda")
        return [q, kv], lambda s: si.sparse_attention(q, kv, idx, stream=s)

    return {"window": window, "cache": cache, "top-k": top_k, "sparse": sparse}


def _busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(400_000_000)  # some 0.2 s


@pytest.mark.parametrize("name", list(_attention_calls()))
def test_memory_of_a_call_on_another_stream_is_not_given_out(name):
    """Inputs and outputs that the caller drops while the call waits on its
    stream keep their memory, and a call's outputs do not take memory that work
    of the current stream still uses."""
    x, call = _attention_calls()[name]()
    s = torch.cuda.Stream()
    call(s)
    torch.cuda.synchronize()
    outs = call(s)
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in (*x, *outs)]
    del outs
    torch.cuda.empty_cache()
    _busy(s)
    outs = call(s)
    taken = {t.data_ptr() for t in (*x, *outs)}
    x.clear()
    del outs, call
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    assert not s.query(), "the stream was to be busy still"
    assert not taken & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    # the other way round: the current stream's own memory
    del new
    x, call = _attention_calls()[name]()
    out_sizes = [t.numel() * t.element_size() for t in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in out_sizes]
    taken = {t.data_ptr() for t in held}
    _busy(torch.cuda.current_stream())
    del held
    outs = call(s)
    assert not torch.cuda.current_stream().query(), "the stream was to be busy still"
    assert not taken & {t.data_ptr() for t in outs}
    torch.cuda.synchronize()
    for a, b in zip(outs, call(None)):
        assert torch.equal(a, b)


def test_captured_calls_on_a_side_stream():
    """A step of append and attention on a side stream of a capture, over a
    cache whose units are cut between blocks, and two such graphs replayed at once."""
    g = _gen(70)
    page, D, H, n = 64, 128, 16, 5000
    width = -(-(n + 8) // page)
    pool = _positive(2 * width, 2, page, D, g)
    table = torch.arange(2 * width, dtype=torch.int32).view(2, width).cuda()
    side = torch.cuda.Stream()
    runs = []
    for i in range(2):
        q, k, v = [torch.randn((2, 1, h, D), generator=g).bfloat16().cuda() for h in (H, 2, 2)]
        lens = _i32([n, n - 100 * i]).cuda()
        cache = _cache(pool)

        def step():
            side.wait_stream(torch.cuda.current_stream())
            si.cache_append(cache, k, v, table, lens, stream=side)
            out = si.cache_attention(q, cache, table, lens + 1, stream=side)
            torch.cuda.current_stream().wait_stream(side)
            return out

        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = step()
        runs.append((graph, out, cache, q, lens, (k, v)))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, run in zip(streams, runs):
            with torch.cuda.stream(s):
                run[0].replay()
    torch.cuda.synchronize()
    for _, out, cache, q, lens, _ in runs:
        now = [t.cpu() for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)]
        want = kv_bounds.cache_attention(q.cpu(), *now, table.cpu(), lens.cpu() + 1)
        kv_bounds.check(*out, want, sharp=None)
    assert si.device_status() == si.SI_OK


# ------------------------------------------------------------------ sizes that a server meets beside decoding


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("L,H,G,D,page,window,n_sink", [
    (300, 8, 2, 64, 16, 0, 0),      # a part of a prompt over a cached prefix
    (300, 8, 2, 64, 16, 100, 5),
    (130, 6, 1, 128, 128, 33, 0),   # more than a tile of queries, three rows of heads a tile's edge
    (17, 5, 5, 128, 32, 0, 0),
])
def test_cache_attention_of_many_queries(dtype, L, H, G, D, page, window, n_sink):
    """More queries than drafted tokens, sequences shorter than they are, the first of them at the start."""
    g = _gen(L)
    lens = [L, 700, L - 7, 3, 0]
    need = [-(-n // page) for n in lens]
    pool = _positive(sum(need) + 1, G, page, D, g)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    for b, part in enumerate(torch.randperm(sum(need), generator=g).int().split(need)):
        table[b, : need[b]] = part
    q = (torch.randn((len(lens), L, H, D), generator=g) * 0.5).to(dtype)
    _check_cache(q, pool, table, _i32(lens), window=window, n_sink=n_sink)


def test_cache_attention_key_that_is_nan_reaches_only_those_who_see_it():
    g = _gen(80)
    page, D, H, L, n = 16, 64, 4, 5, 90
    pool = _positive(6, 1, page, D, g)
    table = torch.arange(6, dtype=torch.int32)[None]
    q = (torch.randn((1, L, H, D), generator=g) * 0.5).bfloat16().cuda()
    lens = _i32([n]).cuda()
    for window, at, who in ((0, n - 3, [2, 3, 4]), (20, n - 22, [0, 1, 2])):
        want = si.cache_attention(q, _cache(pool), table.cuda(), lens, window=window)
        bad = pool[0].clone()
        bad[at // page, 0, at % page, 7] = 0xFF
        out, lse = si.cache_attention(q, _cache([bad, *pool[1:]]), table.cuda(), lens, window=window)
        for i in range(L):
            if i in who:
                assert torch.isnan(out[0, i]).all() and torch.isnan(lse[0, i]).all()
            else:
                assert torch.equal(out[0, i], want[0][0, i]) and torch.equal(lse[0, i], want[1][0, i])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G,window,n_sink", [(8, 1, 128, 4), (6, 2, 250, 0), (4, 4, 350, 30), (16, 1, 600, 3), (3, 1, 900, 0)])
def test_window_attention_to_its_bounds(dtype, D, H, G, window, n_sink):
    """The narrow form and both tile sizes, padded: outputs whose sums do not cancel."""
    g = _gen(window)
    q, k, v = [torch.randn((2, 800, n, D), generator=g) for n in (H, G, G)]
    _check_window(q.to(dtype), k.to(dtype), (v.abs() + 0.1).to(dtype), window, n_sink, _i32([800, 611]))


def test_chunks_of_a_prompt_equal_the_whole():
    """A prompt through the window at once, and in parts through the cache: the
    same where the cache holds the values exactly."""
    g = _gen(81)
    S, H, G, D, page, W, K = 400, 8, 2, 128, 32, 90, 4
    code = torch.randint(0, 256, (2, 1, S, G, D), generator=g, dtype=torch.int16)
    code = torch.where(code % 128 > 0x50, code - 0x38, code).to(torch.uint8)
    k, v = [c.view(torch.float8_e4m3fn).bfloat16().cuda() for c in code]
    # (one magnitude of 448 in each page and head fixes its scale at 1)
    k[:, ::page, :, 0] = v[:, ::page, :, 1] = 448.0
    q = (torch.randn((1, S, H, D), generator=g) * 0.02).bfloat16().cuda()
    want = kv_bounds.window_attention(q.cpu(), k.cpu(), v.cpu(), W, K)
    kv_bounds.check(*si.window_attention(q, k, v, window=W, n_sink=K), want, sharp=None)
    n = -(-S // page)
    pool = [torch.zeros((n, G, page, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pool += [torch.zeros((n, G), device="cuda") for _ in range(2)]
    cache, table = si.PagedCache(*pool), torch.arange(n, dtype=torch.int32, device="cuda")[None]
    done = 0
    for part in (32, 1, 95, 2, 126, 144):  # (the parts that begin a page bring its 448)
        lens = _i32([done]).cuda()
        rows = slice(done, done + part)
        si.cache_append(cache, k[:, rows].contiguous(), v[:, rows].contiguous(), table, lens)
        out, lse = si.cache_attention(q[:, rows].contiguous(), cache, table, lens + part, window=W, n_sink=K)
        see = kv_bounds.visible(torch.arange(done, done + part)[:, None], torch.arange(done + part), W, K)
        ref = kv_bounds.attend(q[0, rows].cpu(), k[0, : done + part].cpu(), v[0, : done + part].cpu(), see, D ** -0.5,
                               *kv_bounds.CACHE[torch.bfloat16], 2.0 ** -8, torch.ones(done + part, G))
        kv_bounds.check(out[0], lse[0], ref, sharp=None)
        done += part
    assert done == S and pool[2].eq(1).all() and pool[3].eq(1).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,page,H,L,window", [
    (64, 16, 2, 4, 0), (128, 16, 4, 4, 50), (64, 32, 8, 4, 60), (128, 64, 16, 4, 0), (64, 128, 128, 2, 200), (128, 16, 5, 40, 20)])
def test_cache_attention_values_that_are_nan(dtype, D, page, H, L, window):
    """NaN values of tokens that some queries see and others do not, for all
    numbers of rows: NaN in those rows' dims, and nothing else changes."""
    g = _gen(D + H)
    n = 300
    n_pages = -(-n // page)
    pool = _positive(n_pages, 1, page, D, g)
    table = torch.randperm(n_pages, generator=g).int()[None]
    q = (torch.randn((1, L, H, D), generator=g) * 0.5).to(dtype).cuda()
    lens = _i32([n]).cuda()
    want = si.cache_attention(q, _cache(pool), table.cuda(), lens, window=window)
    bad = pool[1].clone()
    first = n - L - window + 1 if window else n - L - 5  # (the first query's window begins there)
    where = [(first + i, (13 * i) % D) for i in (-1, 0, 1, 2)] + [(n - 2, 1), (n - 2, D - 1), (n - 1, 16), (n - L, 17)]
    for t, d in where:
        bad[table[0, t // page], 0, t % page, d] = 0x7F if t % 2 else 0xFF
    out, lse = si.cache_attention(q, _cache([pool[0], bad, *pool[2:]]), table.cuda(), lens, window=window)
    assert torch.equal(lse, want[1])
    for i in range(L):
        p = n - L + i
        dims = sorted({d for t, d in where if t <= p and (not window or t > p - window)})
        keep = [d for d in range(D) if d not in dims]
        assert torch.isnan(out[0, i][:, dims]).all()
        assert torch.equal(out[0, i][:, keep], want[0][0, i][:, keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_the_most_heads_that_share_one(dtype):
    """128 query heads on one, through both attentions."""
    g = _gen(90)
    q, k, v = [torch.randn((1, 300, n, 64), generator=g) for n in (128, 1, 1)]
    for window, n_sink in ((100, 3), (280, 0)):
        _check_window(q[:, :150].to(dtype).contiguous(), k[:, :150].to(dtype).contiguous(),
                      (v.abs() + 0.1)[:, :150].to(dtype).contiguous(), window, n_sink)
    pool = _positive(40, 1, 32, 64, g)
    table = torch.arange(40, dtype=torch.int32)[None]
    _check_cache((q[:, :2] * 0.5).to(dtype).contiguous(), pool, table, _i32([1270]), window=0)


@pytest.mark.parametrize("window", [40, 300])
@pytest.mark.parametrize("by_keys", [False, True])
def test_window_attention_scores_that_are_infinite(window, by_keys):
    """A key with an infinity: rows whose score with it is +infinity give NaN,
    those with -infinity do not count it, also in blocks done key by key."""
    g = _gen(91)
    S, at = 500, 100
    q, k, v = [torch.randn((1, S, n, 128), generator=g).bfloat16() for n in (2, 1, 1)]
    q[..., 5] = torch.where(torch.arange(S) % 2 == 0, 1.0, -1.0)[None, :, None]
    v = v.abs() + 0.1
    pos = torch.arange(S)
    see = kv_bounds.visible(pos[:, None], pos, window, 0)
    sees_it = see[:, at]
    k[0, at, 0, 5] = 0
    want = kv_bounds.attend(q[0], k[0], v[0], see & (pos != at), 128 ** -0.5, *kv_bounds.WINDOW[torch.bfloat16], 2.0 ** -8)
    k[0, at, 0, 5] = float("inf")
    if by_keys:  # a value that is NaN, of the last token alone and of one far from the key
        v[0, S - 1, 0, 3] = v[0, at + 30, 0, 3] = float("nan")
    out, lse = [t[0].cpu() for t in si.window_attention(*_cuda(q, k, v), window=window)]
    up = sees_it & (pos % 2 == 0)
    assert torch.isnan(out[up]).all() and torch.isnan(lse[up]).all()
    rest = ~up
    if by_keys:
        touched = see[:, at + 30] | (pos == S - 1)
        assert torch.isnan(out[touched][..., 3]).all()
        out[touched] = torch.where(torch.arange(128) == 3, want[0][touched].bfloat16(), out[touched])
    kv_bounds.check(out[rest], lse[rest], [t[rest] for t in want])
