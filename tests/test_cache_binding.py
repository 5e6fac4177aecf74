"""Refusals of the K/V-cache binding that need no GPU."""
import types

import pytest

import streaming_top_b200 as si


def test_a_stream_of_another_device_is_refused():
    there = types.SimpleNamespace(cuda_stream=0, device_index=1, device="cuda:1")
    with pytest.raises(ValueError, match="stream"):
        si._enqueue("a call", 0, there, lambda s: pytest.fail("enqueued"))
