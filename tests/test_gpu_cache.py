"""The paged 8-bit K/V cache on a GPU: appending, page management, attention
over it, the windowed prompt attention, and a run of them as a server would
make it, against the plain 64-bit forms of tests/kv_reference.py (tolerances
derived there)."""
import random

import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

import streaming_top_b200 as si  # noqa: E402

STEP = {"cache": 2.0 ** -8, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _pool(n_pages, H, page, D, g, nan_every=0):
    """Codes and scales on the CPU; every byte value but the NaN codes."""
    def codes():
        c = torch.randint(0, 256, (n_pages, H, page, D), generator=g, dtype=torch.int16)
        c = torch.where(c % 128 > 0x70, c - 0x38, c)  # most of the range, the largest values rarer
        return c.to(torch.uint8)

    def scales():
        return torch.exp2(torch.randint(-9, -4, (n_pages, H), generator=g).float()) * (
            1 + torch.rand((n_pages, H), generator=g))

    return codes(), codes(), scales(), scales()


def _cuda(*ts):
    return [t.cuda() for t in ts]


def _table(lens, width, page, n_pages, g):
    order = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for j in range(-(-max(n, 0) // page)):
            table[b, j] = order.pop()
    return table


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


# ------------------------------------------------------------------ append


def _run_append(pool, k, v, table, lens, n_new):
    dev = _cuda(*pool)
    cache = si.PagedCache(*dev)
    si.cache_append(cache, k.cuda(), v.cuda(), table.cuda(), lens.cuda(), n_new=None if n_new is None else n_new.cuda())
    full = torch.full_like(lens, k.shape[1]) if n_new is None else n_new
    for codes, scales, dc, ds, x in ((pool[0], pool[2], dev[0], dev[2], k), (pool[1], pool[3], dev[1], dev[3], v)):
        wc, ws = ref.append(codes, scales, x, table, lens, full)
        assert torch.equal(ds.cpu(), ws)
        assert torch.equal(_canonical(dc.cpu()), _canonical(wc))
    return dev


def _canonical(codes):
    """NaN has two codes."""
    return torch.where((codes & 0x7F) == 0x7F, 0x7F, codes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (128, 128), (64, 32)])
@pytest.mark.parametrize("lens,L,n_new", [
    ([0, 5, 31, 200], 1, None),              # decode: first slots, middles, a page's last slot
    ([0, 17, 16, 130], 77, [77, 0, 1, 50]),  # ragged prompts that begin inside a page, one without rows
    ([0, 3, 64, 128], 300, [300, 299, 500, -4]),  # several pages; counts outside [0, L]
])
def test_append(dtype, D, page, lens, L, n_new):
    g = _gen(len(lens) * 100 + L + D + page)
    H = 3
    width = -(-(max(lens) + L) // page) + 1
    total = [a + L for a in lens]
    n_pages = sum(-(-t // page) for t in total) + 3
    pool = _pool(n_pages, H, page, D, g)
    table = _table(total, width, page, n_pages, g)
    k = torch.randn((4, L, H, D), generator=g) * torch.exp(3 * torch.randn((4, L, H, 1), generator=g))
    v = torch.randn((4, L, H, D), generator=g)
    _run_append(pool, k.to(dtype), v.to(dtype), table, _i32(lens), None if n_new is None else _i32(n_new))


def test_append_special_values():
    """Zeros, subnormals, infinities, NaN, values at the scale's border, and a zero and an odd old scale."""
    g = _gen(1)
    page, H, D, L = 16, 1, 64, 8
    pool = _pool(8, H, page, D, g)
    table = _i32([[0, 1], [2, 3], [4, 5], [6, 7]])
    lens = _i32([0, 4, 0, 10])
    k = torch.randn((4, L, H, D), generator=g)
    k[0] = 0
    k[1] *= 1e-39                  # bf16 subnormals: the scale stays a normal number
    k[2, 0, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 3.0e38])
    k[3] = 448.0
    v = torch.zeros((4, L, H, D))
    v[1] = 448.0 * 2.0 ** -20      # exactly at the border of a power of two
    v[2] = 449.0 * 2.0 ** -20
    v[3, 0, 0, 0] = float("inf")   # nothing finite but zeros
    pool[2][2] = 0.0               # the older tokens' scale: all of them zero
    pool[3][6] = 0.7               # not a power of two, and large enough to stay
    _run_append(pool, k.bfloat16(), v.bfloat16(), table, lens, None)


def test_append_drops_what_has_no_page():
    g = _gen(2)
    pool = _pool(4, 2, 16, 128, g)
    table = _i32([[0, -1, 1], [2, 99, -5], [3, 3, 3]])
    lens = _i32([10, 0, -7])       # across a missing page; ids out of range; negative positions
    x = torch.randn((3, 40, 2, 128), generator=g).bfloat16()
    table[2] = _i32([3, -1, -1])
    _run_append(pool, x, -x, table, lens, None)
    # past the end of the table
    _run_append(pool, x[:1], x[:1], _i32([[1, 2]]), _i32([20]), None)


def test_append_twice_equals_once_where_pages_do_not_meet():
    g = _gen(3)
    page, H, D = 32, 2, 128
    pool = _pool(6, H, page, D, g)
    x = torch.randn((1, 64, H, D), generator=g).bfloat16()
    table = _i32([[4, 2, 0]])
    a = _run_append(pool, x, x, table, _i32([0]), None)
    b = _cuda(*pool)
    cache = si.PagedCache(*b)
    for at in (0, 32):
        rows = x[:, at: at + 32].contiguous().cuda()
        si.cache_append(cache, rows, rows, table.cuda(), _i32([at]).cuda())
    for s, t in zip(a, b):
        assert torch.equal(s, t)


# ------------------------------------------------------------------ pages


def _state(n_seq, width, n_pages, page, g, fill=0.6):
    """A random state that shares pages: (table, lens, refs) as lists."""
    rng = random.Random(int(torch.randint(0, 1 << 30, (1,), generator=g)))
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, lens = [[-1] * width for _ in range(n_seq)], [0] * n_seq
    for b in range(n_seq):
        if rng.random() < 0.25:
            continue
        n = rng.randint(1, width * page)
        need = -(-n // page)
        first = [p for p in table[rng.randrange(n_seq)] if p >= 0][: rng.randint(0, need)] if rng.random() < 0.4 else []
        if len(ids) - (need - len(first)) < n_pages * (1 - fill):
            continue
        table[b] = (first + [ids.pop() for _ in range(need - len(first))] + [-1] * width)[:width]
        lens[b] = n
    refs = [0] * n_pages
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    return table, lens, refs


def _same(t, v):
    assert t.cpu().tolist() == v


def _moved_pool(pool, copies):
    out = [t.clone() for t in pool]
    for t, s in zip(out, pool):
        for a, b in copies:
            t[b] = s[a]
    return out


SIZES = [(1, 1, 1, 16), (5, 7, 40, 16), (40, 12, 300, 64), (130, 33, 5000, 16), (600, 5, 2100, 32)]


@pytest.mark.parametrize("n_seq,width,n_pages,page", SIZES)
@pytest.mark.parametrize("share", [True, False])
def test_fork(n_seq, width, n_pages, page, share):
    g = _gen(n_seq * 7 + width)
    pool = _pool(n_pages, 1, page, 64, g)
    table, lens, refs = _state(n_seq, width, n_pages, page, g)
    rng = random.Random(n_seq)
    n = min(n_seq, 77)
    src = [rng.randrange(-1, n_seq + 1) for _ in range(n)]
    dst = [rng.randrange(-1, n_seq + 1) for _ in range(n)]  # some taken, some twice, some outside
    wt, wl, wr, ws, copies = ref.fork(table, lens, refs, src, dst, page, share)
    dev = _cuda(*pool)
    t, l, r = _cuda(_i32(table), _i32(lens), _i32(refs))
    status = si.cache_fork(si.PagedCache(*dev), t, l, r, _i32(src).cuda(), _i32(dst).cuda(), share=share)
    _same(status, ws)
    _same(t, wt)
    _same(l, wl)
    _same(r, wr)
    for got, want in zip(dev, _moved_pool(pool, copies)):
        assert torch.equal(got.cpu(), want)


def test_page_calls_at_their_largest():
    """8192 rows and pairs, pools of more pages than a block scans at once, pages that run out half way."""
    n_seq, page = 8192, 16
    rng = random.Random(5)
    for n_pages, width in ((30000, 3), (9000, 2)):
        g = _gen(n_pages)
        pool = _pool(n_pages, 1, page, 64, g)
        cache = si.PagedCache(*_cuda(*pool))
        ids = list(range(n_pages))
        rng.shuffle(ids)
        table, lens, refs = [[-1] * width for _ in range(n_seq)], [0] * n_seq, [0] * n_pages
        for b in range(n_seq // 2):
            lens[b] = rng.randint(0, 2 * page)
            for j in range(-(-lens[b] // page)):
                if not ids:
                    break
                table[b][j] = ids.pop()
                refs[table[b][j]] = 1
        src = [rng.randrange(n_seq // 2) for _ in range(n_seq)]
        dst = [n_seq // 2 + i if i < n_seq // 2 else rng.randrange(n_seq) for i in range(n_seq)]
        want = ref.fork(table, lens, refs, src, dst, page, True)
        t, l, r = _cuda(_i32(table), _i32(lens), _i32(refs))
        st = si.cache_fork(cache, t, l, r, _i32(src).cuda(), _i32(dst).cuda())
        _same(st, want[3])
        _same(t, want[0])
        _same(l, want[1])
        _same(r, want[2])
        new = [rng.randint(-1, 2 * page) for _ in range(n_seq)]
        wt, wr, ws = ref.reserve(want[0], want[1], want[2], new, page)
        _same(si.cache_reserve(cache, t, l, r, _i32(new).cuda()), ws)
        _same(t, wt)
        _same(r, wr)
        gone = [b for b in range(n_seq) if rng.random() < 0.5]
        wt, wl, wr = ref.free(wt, want[1], wr, gone)
        si.cache_free(cache, t, l, r, _i32(gone).cuda())
        wt, wr, wu, wm, copies = ref.compact(wt, wr)
        before = [x.cpu() for x in (cache.k_pages, cache.v_scale)]
        used, moved = si.cache_compact(cache, t, r)
        assert used.item() == wu
        _same(moved, wm)
        _same(t, wt)
        _same(r, wr)
        a, b = torch.tensor([c[0] for c in copies]), torch.tensor([c[1] for c in copies])
        for x, y in zip(before, (cache.k_pages, cache.v_scale)):
            x[b] = x[a]
            assert torch.equal(x, y.cpu())


def test_fork_runs_out_of_pages():
    """Pairs in order: the first that does not fit and those behind it fail, except the ones that need nothing."""
    page, n_pages = 16, 10
    table = [[0, 1, 2], [3, -1, -1], [4, 5, -1]] + [[-1] * 3 for _ in range(6)]
    lens = [40, 16, 17] + [0] * 6
    refs = [1] * 6 + [0] * 4
    pool = _pool(n_pages, 2, page, 64, _gen(4))
    src, dst = [0, 2, 0, 1, 0, 3], [3, 4, 5, 6, 7, 8]
    for share in (True, False):
        want = ref.fork(table, lens, refs, src, dst, page, share)
        dev = _cuda(*pool)
        t, l, r = _cuda(_i32(table), _i32(lens), _i32(refs))
        st = si.cache_fork(si.PagedCache(*dev), t, l, r, _i32(src).cuda(), _i32(dst).cuda(), share=share)
        _same(st, want[3])
        _same(t, want[0])
        _same(l, want[1])
        _same(r, want[2])
        for got, w in zip(dev, _moved_pool(pool, want[4])):
            assert torch.equal(got.cpu(), w)
    assert want[3] == [0, 1, 1, 1, 1, 0]


@pytest.mark.parametrize("n_seq,width,n_pages,page", SIZES)
def test_reserve(n_seq, width, n_pages, page):
    g = _gen(n_seq * 3 + width)
    pool = _pool(n_pages, 1, page, 64, g)
    table, lens, refs = _state(n_seq, width, n_pages, page, g)
    rng = random.Random(n_seq + 1)
    new = [rng.choice([0, -3, 1, page, rng.randint(1, width * page), 2 ** 31 - 1 - max(lens)]) for _ in range(n_seq)]
    wt, wr, ws = ref.reserve(table, lens, refs, new, page)
    t, l, r = _cuda(_i32(table), _i32(lens), _i32(refs))
    st = si.cache_reserve(si.PagedCache(*_cuda(*pool)), t, l, r, _i32(new).cuda())
    _same(st, ws)
    _same(t, wt)
    _same(r, wr)


@pytest.mark.parametrize("n_seq,width,n_pages,page", SIZES)
def test_free_then_compact(n_seq, width, n_pages, page):
    g = _gen(n_seq * 5 + width)
    pool = _pool(n_pages, 1, page, 64, g)
    table, lens, refs = _state(n_seq, width, n_pages, page, g)
    rng = random.Random(n_seq + 2)
    rows = [rng.randrange(-2, n_seq + 2) for _ in range(n_seq // 2 + 1)] * 2  # rows twice, rows outside
    wt, wl, wr = ref.free(table, lens, refs, rows)
    dev = _cuda(*pool)
    cache = si.PagedCache(*dev)
    t, l, r = _cuda(_i32(table), _i32(lens), _i32(refs))
    si.cache_free(cache, t, l, r, _i32(rows).cuda())
    _same(t, wt)
    _same(l, wl)
    _same(r, wr)
    wt, wr, wu, wm, copies = ref.compact(wt, wr)
    used, moved = si.cache_compact(cache, t, r)
    assert used.item() == wu
    _same(moved, wm)
    _same(t, wt)
    _same(r, wr)
    for got, want in zip(dev, _moved_pool(pool, copies)):
        assert torch.equal(got.cpu(), want)
    used, moved = si.cache_compact(cache, t, r)  # once more: nothing moves
    assert used.item() == wu
    _same(t, wt)


# ------------------------------------------------------------------ attention over the cache


def _run_cache(pool, q, table, lens, window=0, n_sink=0, scale=0.0, **kw):
    dev = _cuda(*pool)
    out, lse = si.cache_attention(q.cuda(), si.PagedCache(*dev), table.cuda(), lens.cuda(), window=window,
                                  n_sink=n_sink, scale=scale, **kw)
    assert si.device_status() == si.SI_OK
    return out, lse


def _check_cache(pool, q, table, lens, window=0, n_sink=0, scale=0.0):
    got = _run_cache(pool, q, table, lens, window, n_sink, scale)
    want = ref.cache_attention(q, *pool, table, lens, window, n_sink, scale)
    page = pool[0].shape[2]
    ids = table[(table >= 0) & (table < pool[0].shape[0])].long()
    vmax = ref.dequantise(pool[1][ids], pool[3][ids]).nan_to_num().abs().max().item() if len(ids) else 0.0
    ref.check(got, want, STEP["cache"], vmax, min(int(lens.max()), table.shape[1] * page))
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L,H,G,page,lens,window,n_sink", [
    (1, 8, 1, 16, [1, 0, 15, 16, 17], 0, 0),       # lengths zero and one, page borders
    (1, 8, 8, 64, [127, 128, 129, 300], 0, 0),     # a head each; tile borders
    (1, 64, 1, 128, [700], 0, 0),                  # 64 heads on one
    (1, 6, 2, 32, [1000, 3, 257], 0, 0),           # three heads on one
    (3, 8, 2, 16, [2, 1, 0, 200, 130], 0, 0),      # fewer tokens than queries
    (4, 20, 4, 32, [64, 129, 511], 33, 2),         # window and sinks, five heads on one, odd sizes
    (1, 16, 2, 16, [1500, 40, 1], 128, 4),
    (2, 4, 2, 64, [900, 131, 385], 1, 0),          # a window of one token
    (1, 4, 2, 16, [600, 250], 16, 200),            # many sinks, their tile apart from the window's or next to it
    (5, 130, 2, 16, [333, 7], 100, 130),           # 325 rows a key/value head
])
def test_cache_attention(dtype, D, L, H, G, page, lens, window, n_sink):
    g = _gen(L * 1000 + H * 10 + page)
    width = -(-max(lens) // page) + 1
    n_pages = sum(-(-n // page) for n in lens) + 2
    pool = _pool(n_pages, G, page, D, g)
    table = _table(lens, width, page, n_pages, g)
    q = (torch.randn((len(lens), L, H, D), generator=g) * 0.5).to(dtype)
    _check_cache(pool, q, table, _i32(lens), window, n_sink)


def test_cache_attention_of_a_long_context():
    """More tiles than a launch has blocks, and lengths that differ by a factor of thousands."""
    g = _gen(11)
    lens = [60000, 13, 4000]
    page, G, D, H = 64, 1, 128, 2
    n_pages = sum(-(-n // page) for n in lens)
    pool = _pool(n_pages, G, page, D, g)
    table = _table(lens, -(-max(lens) // page), page, n_pages, g)
    q = torch.randn((3, 1, H, D), generator=g).bfloat16()
    _check_cache(pool, q, table, _i32(lens))
    _check_cache(pool, q, table, _i32(lens), scale=0.01)


def test_cache_attention_ignores_what_nobody_sees():
    """NaN codes and NaN scales in slots behind the end, before the window, in
    unused and missing pages; entries out of range."""
    g = _gen(12)
    page, G, D, H = 16, 2, 128, 8
    pool = list(_pool(40, G, page, D, g))
    lens = _i32([37, 100, 20])
    table = _table([37, 100, 20], 8, page, 30, g)
    table[2, 0] = -1
    table[1, 3] = 1000
    for b, n in enumerate([37, 100, 20]):
        last = int(table[b, (n - 1) // page])
        for t in pool[:2]:
            t[last, :, n % page or page:] = 0x7F
    for t in pool[:2]:
        t[30:] = 0xFF
    pool[2][30:] = float("nan")
    pool[3][30:] = float("inf")
    table[:, 7] = 35
    q = torch.randn((3, 1, H, D), generator=g).bfloat16()
    _check_cache(pool, q, table, lens)
    # before the window: the first page's tokens but the sinks
    first = int(table[1, 0])
    for t in pool[:2]:
        t[first, :, 2:] = 0x7F
    _check_cache(pool, q[1:2], table[1:2], lens[1:2], window=50, n_sink=2)


def test_cache_attention_nan_reaches_only_those_who_see_it():
    """The last token's value holds NaN in some dims: earlier queries of the
    same call do not see it; the last one does, in those dims."""
    g = _gen(13)
    page, G, D, H, L = 16, 1, 128, 4, 3
    pool = list(_pool(4, G, page, D, g))
    table = _i32([[2, 0, 3]])
    n = 40
    clean = torch.randn((1, L, H, D), generator=g).bfloat16()
    want = _run_cache(pool, clean, table, _i32([n]))
    pool[1] = pool[1].clone()
    pool[1][3, 0, (n - 1) % page, 5] = 0x7F
    pool[1][3, 0, (n - 1) % page, 77] = 0xFF
    got = _run_cache(pool, clean, table, _i32([n]))
    assert torch.equal(got[0][:, :2], want[0][:, :2])
    nan = torch.isnan(got[0][:, 2])
    assert nan[..., [5, 77]].all() and nan.sum() == 2 * H
    assert torch.equal(got[1], want[1])


def test_cache_attention_lengths_beyond_the_table():
    g = _gen(14)
    pool = _pool(6, 1, 16, 64, g)
    table = _i32([[0, 1], [2, 3], [4, 5]])
    q = torch.randn((3, 1, 2, 64), generator=g).half()
    _check_cache(pool, q, table, _i32([1000, -5, 32]))
    _check_cache(pool, q, table, _i32([2 ** 31 - 1, -2 ** 31, 31]), window=2 ** 31 - 1, n_sink=2 ** 31 - 1)
    _check_cache(pool, q, table, _i32([32, 16, 1]), window=2 ** 31 - 1, n_sink=0)


def test_cache_attention_scales_far_apart():
    """Value scales that differ by 2^24 between pages, one of them zero."""
    g = _gen(15)
    page = 16
    pool = list(_pool(20, 1, page, 128, g))
    pool[3] = torch.exp2(torch.randint(-12, 13, (20, 1), generator=g).float())
    pool[3][3] = 0.0
    pool[2][5] = 0.0
    table = _table([300], 19, page, 20, g)
    q = torch.randn((1, 1, 8, 128), generator=g).bfloat16()
    _check_cache(pool, q, table, _i32([300]))


def test_cache_attention_extreme_scores():
    """Scores in the thousands: one token takes all the weight; large and tiny queries."""
    g = _gen(16)
    pool = _pool(12, 1, 16, 128, g)
    table = _table([150], 10, 16, 12, g)
    for mag in (2.0 ** -100, 1e-3, 100.0, 1e4):
        q = (torch.randn((1, 1, 4, 128), generator=g) * mag).bfloat16()
        out, lse = _run_cache(pool, q, table, _i32([150]))
        want = ref.cache_attention(q, *pool, table, _i32([150]))
        if mag < 100:
            ref.check((out, lse), want, STEP["cache"], 448.0, 150)
        else:  # the scores' own rounding exceeds 1: the largest score still shows in lse
            assert torch.isfinite(out).all()
            assert torch.allclose(lse.cpu().double(), want[1], rtol=2 ** -14)


# ------------------------------------------------------------------ prompts


def _check_window(q, k, v, window, n_sink=0, lens=None, scale=0.0, poison=False):
    if poison and lens is not None:
        for b, n in enumerate(lens.tolist()):
            q[b, max(n, 0):] = float("nan")
            k[b, max(n, 0):] = float("nan")
            v[b, max(n, 0):] = float("inf")
    qd, kd, vd = _cuda(q, k, v)
    got = si.window_attention(qd, kd, vd, window=window, n_sink=n_sink, lens=None if lens is None else lens.cuda(),
                              scale=scale)
    assert si.device_status() == si.SI_OK
    want = ref.window_attention(q, k, v, window, n_sink, lens, scale)
    vmax = v.double()[torch.isfinite(v)].abs().max().item()
    ref.check(got, want, STEP[q.dtype], vmax, min(q.shape[1], window + n_sink))
    return got


def _qkv(B, S, H, G, D, dtype, seed):
    g = _gen(seed)
    return [torch.randn((B, S, n, D), generator=g).to(dtype) for n in (H, G, G)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,S,H,G,window,n_sink", [
    (1, 1, 1, 1, 1, 0),
    (2, 7, 4, 2, 3, 1),
    (1, 130, 4, 4, 128, 0),      # one row past a tile
    (1, 300, 8, 1, 128, 4),
    (1, 257, 6, 2, 64, 70),      # three heads on one; more sinks than window
    (1, 400, 2, 1, 1, 0),        # each token sees itself
    (1, 400, 2, 2, 400, 0),      # plain causal
    (1, 390, 5, 1, 17, 3),       # five heads on one
    (1, 520, 2, 1, 200, 129),    # sinks past a tile
])
def test_window_attention(dtype, D, B, S, H, G, window, n_sink):
    q, k, v = _qkv(B, S, H, G, D, dtype, S + H)
    _check_window(q, k, v, window, n_sink)


@pytest.mark.parametrize("H,G", [(64, 1), (130, 2), (7, 7)])
def test_window_attention_head_layouts(H, G):
    q, k, v = _qkv(1, 70, H, G, 64, torch.bfloat16, H)
    _check_window(q, k, v, 33, 2)


def test_window_attention_padded():
    lens = _i32([0, 1, 129, 250, 300, -3])
    q, k, v = _qkv(6, 250, 4, 2, 128, torch.bfloat16, 5)
    _check_window(q, k, v, 100, 3, lens, poison=True)


def test_window_attention_nan_outside_the_window():
    """NaN and infinities before the window reach nobody past it, nor do later
    tokens: the rows that do not see them stay within the tolerance of the
    clean inputs' exact rows.  (They need not equal the clean call's bits: a
    block with such values is computed key by key, with unrounded weights.)"""
    q, k, v = _qkv(1, 300, 2, 1, 128, torch.bfloat16, 6)
    want = ref.window_attention(q, k, v, 40, 2)
    qd, kd, vd = _cuda(q, k, v)
    kd[0, 100] = float("nan")
    vd[0, 101] = float("inf")
    vd[0, 102, 0, 3] = float("nan")
    got = si.window_attention(qd, kd, vd, window=40, n_sink=2)
    assert si.device_status() == si.SI_OK
    ok = torch.ones(300, dtype=torch.bool)
    ok[100:142] = False
    ref.check([t[:, ok.cuda()] for t in got], [t[:, ok] for t in want], STEP[torch.bfloat16], v.abs().max().item(), 42)
    assert torch.isnan(got[0][0, 100:140]).all()
    # row 140 sees keys 101 .. 140: infinity everywhere, NaN in the one dim of key 102
    dims = torch.arange(128, device="cuda") != 3
    assert torch.isnan(got[0][0, 140, :, 3]).all() and torch.isinf(got[0][0, 140][:, dims]).all()


def test_window_attention_extremes():
    q, k, v = _qkv(1, 200, 2, 1, 64, torch.float16, 7)
    _check_window(q, k, v, 2 ** 31 - 1, 2 ** 31 - 1)
    _check_window(q * 0, k, v, 50, 0, scale=3.0)
    out, lse = si.window_attention(*_cuda(q * 60, k * 60, v), window=50)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


# ------------------------------------------------------------------ as a server uses them


def test_prompt_then_decode_with_forks_and_compaction():
    """Prompts through the window, their rows into the cache, decode steps of
    the sequences and their forks over it, some of them freed and the pages
    moved together: every step equals the plain form on the same cache, and
    what a sequence sees does not change when its pages move."""
    g = _gen(20)
    page, G, H, D, W, K = 16, 2, 8, 128, 40, 3
    n_seq, width, n_pages = 6, 12, 64
    pool = _cuda(*_pool(n_pages, G, page, D, g))
    cache = si.PagedCache(*pool)
    table = torch.full((n_seq, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    new = _i32([70, 33, 100, 0, 0, 0]).cuda()
    q, k, v = _cuda(*_qkv(n_seq, 100, H, G, D, torch.bfloat16, 21))
    _check_window(q.cpu(), k.cpu(), v.cpu(), W, K, new.cpu())
    assert si.cache_reserve(cache, table, lens, refs, new).eq(0).all()
    si.cache_append(cache, k, v, table, lens, n_new=new)
    lens += new
    st = si.cache_fork(cache, table, lens, refs, _i32([0, 2, 0]).cuda(), _i32([3, 4, 5]).cuda())
    assert st.eq(0).all()
    for step in range(20):
        q, k, v = _cuda(*_qkv(n_seq, 1, H, G, D, torch.bfloat16, 30 + step))
        one = torch.ones_like(lens)
        assert si.cache_reserve(cache, table, lens, refs, one).eq(0).all()
        si.cache_append(cache, k, v, table, lens)
        lens += 1
        out, lse = si.cache_attention(q, cache, table, lens, window=W, n_sink=K)
        if step % 7 == 0:
            cpu = [t.cpu() for t in pool]
            want = ref.cache_attention(q.cpu(), *cpu, table.cpu(), lens.cpu(), W, K)
            ref.check((out, lse), want, STEP["cache"], 448.0 * cpu[3].max().item(), W + K)
        if step == 9:
            # the forks share full pages and own their last one
            t = table.cpu()
            assert t[0, 0] == t[3, 0] == t[5, 0] and len({int(t[i, 4]) for i in (0, 3, 5)}) == 3
    si.cache_free(cache, table, lens, refs, _i32([1, 0]).cuda())
    before = si.cache_attention(q, cache, table, lens, window=W, n_sink=K)
    used, moved = si.cache_compact(cache, table, refs)
    assert int(table.max()) < used.item() and int((refs > 0).sum()) == used.item()
    after = si.cache_attention(q, cache, table, lens, window=W, n_sink=K)
    for a, b in zip(before, after):
        assert torch.equal(a, b)


def test_capture_and_replay():
    """A decode step captured once and replayed on new values; two graphs in turn."""
    g = _gen(22)
    page, G, H, D = 64, 2, 16, 128
    lens0 = [500, 900, 64]
    n_pages = 40
    pool = _cuda(*_pool(n_pages, G, page, D, g))
    cache = si.PagedCache(*pool)
    table = _table([n + 64 for n in lens0], 16, page, n_pages, g).cuda()
    lens = _i32(lens0).cuda()
    q, k, v = _cuda(*_qkv(3, 1, H, G, D, torch.bfloat16, 23))

    def step():
        si.cache_append(cache, k, v, table, lens)
        lens.add_(1)
        return si.cache_attention(q, cache, table, lens)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            graphs.append((gr, step()))
    lens.copy_(_i32(lens0))
    for i in range(6):
        for t, n in zip((q, k, v), (H, G, G)):
            t.copy_(torch.randn((3, 1, n, D), generator=g))
        gr, (out, lse) = graphs[i % 2]
        gr.replay()
        want = ref.cache_attention(q.cpu(), *[t.cpu() for t in pool], table.cpu(), lens.cpu())
        ref.check((out, lse), want, STEP["cache"], 448.0 * pool[3].max().item(), 1000)


def test_calls_on_two_streams_at_once():
    g = _gen(24)
    page, G, H, D = 64, 1, 32, 128
    pool = _pool(200, G, page, D, g)
    dev = _cuda(*pool)
    cache = si.PagedCache(*dev)
    table = _table([6000, 5000], 100, page, 200, g).cuda()
    lens = _i32([6000, 5000]).cuda()
    q = torch.randn((2, 1, H, D), generator=g).bfloat16().cuda()
    want = si.cache_attention(q, cache, table, lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(10):
        for s in streams:
            got.append(si.cache_attention(q, cache, table, lens, stream=s))
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_refusals_leave_the_context_usable():
    q = torch.zeros((1, 1, 2, 96), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(si.SIError) as e:
        si.window_attention(q, q, q, window=4)
    assert e.value.status == si.SI_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        si.window_attention(q.transpose(1, 2), q, q, window=4)
    pool = _cuda(*_pool(4, 1, 16, 64, _gen(1)))
    cache = si.PagedCache(*pool)
    t, l, r = _cuda(_i32([[0, 1]]), _i32([20]), _i32([1, 1, 0, 0]))
    si.test_fail_allocations(1)
    with pytest.raises(si.SIError) as e:
        si.cache_reserve(cache, t, l, r, _i32([20]).cuda())
    assert e.value.status == si.SI_ERR_OUT_OF_MEMORY
    assert si.cache_reserve(cache, t, l, r, _i32([10]).cuda()).item() == 0


def test_offsets_past_32_bits():
    """Pools of more than 2^32 bytes: append, attention, fork and compaction at their far end."""
    g = _gen(31)
    page, G, D, H, n = 128, 8, 128, 16, 300
    n_pages = (1 << 32) // (G * page * D) + 40
    kp = torch.zeros((n_pages, G, page, D), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    ks, vs = [torch.zeros((n_pages, G), device="cuda") for _ in range(2)]
    cache = si.PagedCache(kp, vp, ks, vs)
    table = _i32([[n_pages - 1, n_pages - 7, n_pages - 3, -1], [-1] * 4]).cuda()
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[0, :3].long()] = 1
    refs[: n_pages - 20] = 1  # all but the last pages are taken
    x = torch.randn((2, n, G, D), generator=g).bfloat16().cuda()
    lens = _i32([0, 0]).cuda()
    si.cache_append(cache, x, -x, table, lens, n_new=_i32([n, 0]).cuda())
    lens = _i32([n, 0]).cuda()
    q = torch.randn((2, 1, H, D), generator=g).bfloat16().cuda()

    def check(out, lse):
        ids = table.unique()
        ids = ids[ids >= 0].long()
        small = torch.searchsorted(ids, table.long()).int()
        small[table < 0] = -1
        pool = [t[ids].cpu() for t in (kp, vp, ks, vs)]
        want = ref.cache_attention(q.cpu(), *pool, small.cpu(), lens.cpu())
        ref.check((out, lse), want, STEP["cache"], 448.0 * pool[3].max().item(), n)

    check(*si.cache_attention(q, cache, table, lens))
    assert si.cache_fork(cache, table, lens, refs, _i32([0]).cuda(), _i32([1]).cuda()).item() == 0
    assert int(table[1, 2]) == n_pages - 20 and int(lens[1]) == n
    a = si.cache_attention(q, cache, table, lens)
    check(*a)
    refs[:4] = 0
    si.cache_compact(cache, table, refs)
    b = si.cache_attention(q, cache, table, lens)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert si.device_status() == si.SI_OK


def test_own_workspace_and_status_word():
    g = _gen(32)
    pool = _cuda(*_pool(60, 2, 64, 128, g))
    cache = si.PagedCache(*pool)
    table = _table([3000], 60, 64, 60, g).cuda()
    lens = _i32([3000]).cuda()
    q = torch.randn((1, 1, 64, 128), generator=g).half().cuda()
    want = si.cache_attention(q, cache, table, lens)
    ws = torch.empty(si.cache_attention_workspace_size(128), dtype=torch.uint8, device="cuda")
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    si.test_fail_allocations(1)  # with its own workspace the call allocates nothing
    got = si.cache_attention(q, cache, table, lens, workspace=ws, device_status=status)
    with pytest.raises(si.SIError):
        si.cache_attention(q, cache, table, lens)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and status.eq(0).all()
    q, k, v = _cuda(*_qkv(1, 100, 4, 2, 64, torch.float16, 33))
    si.window_attention(q, k, v, window=10, device_status=status)
    assert status.eq(0).all()


def test_outputs_aligned_to_16_bytes_only():
    """Slices of a larger buffer, 16 but not 32 bytes aligned."""
    q, k, v = _cuda(*_qkv(1, 300, 4, 2, 64, torch.bfloat16, 34))
    for window in (20, 300):
        want = si.window_attention(q, k, v, window=window)
        flat = torch.full((q.numel() + 16,), 7.0, dtype=q.dtype, device="cuda")
        out = flat[8: 8 + q.numel()].view_as(q)
        assert out.data_ptr() % 32 == 16
        si.window_attention(q, k, v, window=window, out=out)
        assert torch.equal(out, want[0])
        assert (flat[:8] == 7).all() and (flat[-8:] == 7).all()


def test_page_calls_captured():
    """Reserve, fork, free and compact in one graph, replayed from the same state: the same result as eagerly."""
    g = _gen(35)
    page, n_pages = 16, 300
    pool = _cuda(*_pool(n_pages, 2, page, 64, g))
    table, lens, refs = _state(40, 12, n_pages, page, g)
    empty = [b for b in range(40) if lens[b] == 0][:3]
    full = [b for b in range(40) if lens[b] > 0][:3]
    state = _cuda(_i32(table), _i32(lens), _i32(refs))
    work = [t.clone() for t in state]
    src, dst, rows = _cuda(_i32(full), _i32(empty), _i32(full[:1]))
    new = torch.full((40,), 5, dtype=torch.int32, device="cuda")
    cache = si.PagedCache(*pool)

    def step():
        t, l, r = work
        a = si.cache_fork(cache, t, l, r, src, dst)
        b = si.cache_reserve(cache, t, l, r, new)
        si.cache_free(cache, t, l, r, rows)
        return (a, b) + si.cache_compact(cache, t, r)

    first = [t.clone() for t in pool]
    want = [t.clone() for t in step()] + [t.clone() for t in work + pool]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step()
    for _ in range(2):
        for t, v in zip(work + pool, state + first):
            t.copy_(v)
        gr.replay()
        for a, b in zip(list(got) + work + pool, want):
            assert torch.equal(a, b)


def test_many_sequences():
    """More sequences than a block has threads, most of them short, and more units than CTAs."""
    g = _gen(36)
    B, page = 700, 16
    lens = [(7 * b) % 40 for b in range(B)]
    lens[333] = 2500
    n_pages = sum(-(-n // page) for n in lens)
    pool = _pool(n_pages, 2, page, 64, g)
    table = _table(lens, -(-2500 // page), page, n_pages, g)
    q = torch.randn((B, 1, 4, 64), generator=g).bfloat16()
    _check_cache(pool, q, table, _i32(lens))
    _check_cache(pool, q, table, _i32(lens), window=30, n_sink=1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
def test_window_attention_wide(dtype, D):
    """Key tiles of 128, sinks of a tile of their own (20) and of a small one (7), a padded batch."""
    q, k, v = _qkv(2, 900, 4, 1, D, dtype, 40)
    _check_window(q, k, v, 450, 7)
    _check_window(q, k, v, 600, 20, _i32([900, 711]), poison=True)  # (writes NaN into the padding)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window,n_sink,down", [(40, 3, False), (128, 0, False), (300, 0, False), (500, 5, False),
                                                (128, 4, True), (500, 0, True)])
def test_window_attention_scores_that_grow(dtype, window, n_sink, down):
    """Scores that climb by some 40 along the keys (or fall): the running
    maximum leaves its reference again and again, in the narrow form and in
    both tile sizes of the streaming one."""
    g = _gen(41)
    S, H, D = 700, 8, 128
    q = torch.randn((1, S, H, D), generator=g) * 0.05
    k = torch.randn((1, S, 1, D), generator=g) * 0.05
    v = torch.randn((1, S, 1, D), generator=g)
    q[..., 0] = 8.0
    ramp = torch.arange(S) / S
    k[0, :, 0, 0] = 60.0 * (1 - ramp if down else ramp)
    _check_window(q.to(dtype), k.to(dtype), v.to(dtype), window, n_sink)


@pytest.mark.parametrize("down", [False, True])
def test_cache_attention_scores_that_grow(down):
    """The same over a cache of several tiles, cut between CTAs."""
    g = _gen(42)
    page, D, n = 64, 128, 3000
    n_pages = -(-n // page)
    kp, vp, ks, vs = _pool(n_pages, 1, page, D, g)
    table = _table([n], n_pages, page, n_pages, g)
    order = table[0].tolist()
    ks = torch.full((n_pages, 1), 2.0 ** -8)
    for j, p in enumerate(order):  # the first dim's code grows with the page
        x = 400.0 * ((n_pages - 1 - j) if down else j) / n_pages
        kp[p, :, :, 0] = torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn((1, 1, 8, D), generator=g) * 0.1
    q[..., 0] = 200.0
    _check_cache((kp, vp, ks, vs), q.bfloat16(), table, _i32([n]))
