"""Refusals of the K/V-cache and window attention calls: every one is decided
on the host, before any CUDA call, so these run without a GPU on addresses
that nothing reads."""
import ctypes

import pytest
import torch

import streaming_top_b200 as si

P = 4096  # an aligned address; never dereferenced
BAD, UNSUP = si.SI_ERR_INVALID_ARGUMENT, si.SI_ERR_UNSUPPORTED
I31 = 2 ** 31 - 1


def _cache(**kw):
    c = dict(k_pages=P, v_pages=P, k_scale=P, v_scale=P, n_pages=8, H_kv=2, page=16, D=128)
    c.update(kw)
    return ctypes.byref(si._Cache(*c.values()))


CACHE = [({"k_pages": None}, BAD), ({"v_scale": None}, BAD), ({"n_pages": 0}, BAD), ({"H_kv": -1}, BAD),
         ({"k_pages": P + 8}, BAD), ({"k_scale": P + 2}, BAD), ({"page": 24}, UNSUP), ({"page": 256}, UNSUP),
         ({"D": 96}, UNSUP), ({"n_pages": I31, "page": 128}, UNSUP)]


def _append(c=None, k=P, v=P, table=P, lens=P, n_new=None, B=1, L=1, max_pages=4, dtype=0):
    return si.lib().si_cache_append(c or _cache(), k, v, table, lens, n_new, B, L, max_pages, dtype, None)


@pytest.mark.parametrize("kw,status", [
    ({"k": None}, BAD), ({"table": None}, BAD), ({"lens": None}, BAD), ({"B": 0}, BAD), ({"L": -3}, BAD),
    ({"max_pages": 0}, BAD), ({"k": P + 2}, BAD), ({"n_new": P + 1}, BAD), ({"dtype": 1}, UNSUP),
    ({"dtype": 7}, UNSUP), ({"B": I31, "L": 1}, UNSUP)])
def test_append_refuses(kw, status):
    assert _append(**kw) == status
    assert si.lib().si_last_error()


@pytest.mark.parametrize("kw,status", CACHE)
def test_every_call_refuses_a_bad_cache(kw, status):
    c = _cache(**kw)
    L = si.lib()
    assert _append(c) == status
    assert _attend(c) == status
    assert L.si_cache_reserve(c, P, P, P, P, 4, 4, P, None) == status
    assert L.si_cache_fork(c, P, P, P, P, P, 1, 4, 4, 1, P, None) == status
    assert L.si_cache_compact(c, P, P, 4, 4, P, P, None) == status


def test_a_null_cache_is_refused():
    assert si.lib().si_cache_append(None, P, P, P, P, None, 1, 1, 4, 0, None) == BAD
    assert si.lib().si_cache_compact(None, P, P, 4, 4, P, P, None) == BAD


def _attend(c=None, q=P, table=P, lens=P, B=1, L=1, H=4, max_pages=4, window=0, n_sink=0, scale=0.0, dtype=0, out=P,
            lse=P, opt=None):
    return si.lib().si_cache_attention(q, c or _cache(), table, lens, B, L, H, max_pages, window, n_sink, scale, dtype,
                                       out, lse, None, opt)


def _window(q=P, k=P, v=P, lens=None, B=1, S=8, H=4, H_kv=2, D=128, window=4, n_sink=0, scale=0.0, dtype=0, out=P,
            lse=P, opt=None):
    return si.lib().si_window_attention(q, k, v, lens, B, S, H, H_kv, D, window, n_sink, scale, dtype, out, lse, None,
                                        opt)


BOTH = [({"q": None}, BAD), ({"out": None}, BAD), ({"q": P + 4}, BAD), ({"out": P + 8}, BAD), ({"lse": P + 1}, BAD),
        ({"B": 0}, BAD), ({"H": 0}, BAD), ({"n_sink": -1}, BAD), ({"scale": -1.0}, BAD),
        ({"scale": float("nan")}, BAD), ({"scale": float("inf")}, BAD), ({"dtype": 1}, UNSUP), ({"H": 5}, UNSUP),
        ({"H": 2 * 129}, UNSUP), ({"B": I31}, UNSUP)]


@pytest.mark.parametrize("kw,status", BOTH + [({"table": None}, BAD), ({"L": 0}, BAD), ({"max_pages": 0}, BAD),
                                              ({"window": -1}, BAD), ({"lens": P + 2}, BAD)])
def test_cache_attention_refuses(kw, status):
    assert _attend(**kw) == status
    assert si.lib().si_last_error()


@pytest.mark.parametrize("kw,status", BOTH + [({"k": None}, BAD), ({"S": 0}, BAD), ({"window": 0}, BAD),
                                              ({"v": P + 8}, BAD), ({"lens": P + 2}, BAD), ({"D": 96}, UNSUP),
                                              ({"H_kv": 0}, BAD)])
def test_window_attention_refuses(kw, status):
    assert _window(**kw) == status
    assert si.lib().si_last_error()


def test_a_misaligned_status_word_is_refused():
    o = si.Options()
    o.device_status = P + 4
    assert _attend(opt=ctypes.byref(o)) == BAD
    assert _window(opt=ctypes.byref(o)) == BAD


def test_page_calls_refuse():
    L, c = si.lib(), _cache()
    assert L.si_cache_reserve(c, None, P, P, P, 4, 4, P, None) == BAD
    assert L.si_cache_reserve(c, P, P, P, P, 0, 4, P, None) == BAD
    assert L.si_cache_reserve(c, P, P, P, P, 4, 0, P, None) == BAD
    assert L.si_cache_reserve(c, P, P, P, None, 4, 4, P, None) == BAD
    assert L.si_cache_reserve(c, P, P + 2, P, P, 4, 4, P, None) == BAD
    assert L.si_cache_reserve(c, P, P, P, P, 8193, 4, P, None) == UNSUP
    assert L.si_cache_fork(c, P, P, P, P, P, -1, 4, 4, 1, P, None) == BAD
    assert L.si_cache_fork(c, P, P, P, None, P, 1, 4, 4, 1, P, None) == BAD
    assert L.si_cache_fork(c, P, P, P, P, P, 8193, 4, 4, 1, P, None) == UNSUP
    assert L.si_cache_fork(c, P, P, P, None, None, 0, 4, 4, 1, P, None) == si.SI_OK
    assert L.si_cache_free(None, P, P, P, 1, 4, 4, 8, None) == BAD
    assert L.si_cache_free(P, P, P, P, -1, 4, 4, 8, None) == BAD
    assert L.si_cache_free(P, P, P, None, 0, 4, 4, 8, None) == si.SI_OK
    assert L.si_cache_compact(c, P, P, 4, 4, None, P, None) == BAD
    assert L.si_cache_compact(c, P, P, 8193, 4, P, P, None) == UNSUP


def test_binding_refuses_other_tensors():
    z = torch.zeros
    with pytest.raises(ValueError):  # not on a GPU
        si.PagedCache(z(2, 1, 16, 128, dtype=torch.uint8), z(2, 1, 16, 128, dtype=torch.uint8), z(2, 1), z(2, 1))
    with pytest.raises(ValueError):  # not codes
        si.PagedCache(z(2, 1, 16, 128), z(2, 1, 16, 128), z(2, 1), z(2, 1))
    q = z(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        si.window_attention(q, q, q, window=2)
    with pytest.raises(ValueError):
        si.window_attention(q.float(), q, q, window=2)
