"""la2.check(stream) reads the error word of the stream's device, which need not be the
current one (CPU: the device context and the library call are stand-ins)."""

import contextlib
import types

import pytest
import torch

from linear_attention_la2_b200 import build

build.build()

from linear_attention_la2_b200 import la2  # noqa: E402


def test_check_asks_the_streams_device(monkeypatch):
    current, asked = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        try:
            yield
        finally:
            current[0] = before

    def la2_check(stream):
        asked.append((current[0], stream.value))
        return la2.LA2_ERR_INVALID_ARG if current[0] == 1 else la2.LA2_OK

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(la2, "la2_check", la2_check)
    with pytest.raises(la2.La2Error):
        la2.check(types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=7))
    assert asked == [(1, 7)] and current == [0]
