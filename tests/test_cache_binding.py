"""Refusals of the K/V-cache binding that need no GPU."""
import types

import pytest
import torch

import streaming_top_b200 as si


def test_a_stream_of_another_device_is_refused():
    there = types.SimpleNamespace(cuda_stream=0, device_index=1, device="cuda:1")
    with pytest.raises(ValueError, match="stream"):
        si._enqueue("a call", 0, there, lambda s: pytest.fail("enqueued"))


@pytest.mark.parametrize("kw", [{"window": 2 ** 32 + 5}, {"window": 2 ** 31}, {"window": 4, "n_sink": 2 ** 32}])
def test_an_integer_that_would_wrap_is_refused(kw):
    """(A window of 2^32 + 5 would have been one of 5.)"""
    q = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    name = "n_sink" if "n_sink" in kw else "window"
    with pytest.raises(ValueError, match=f"{name} must fit"):
        si.window_attention(q, q, q, **kw)
    with pytest.raises(ValueError, match=f"{name} must fit"):
        si.cache_attention(q, None, None, None, **kw)
