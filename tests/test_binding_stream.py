"""Which stream a binding's call goes to when none is given."""
import types

import torch

from tests.test_kv4_cache import pkg  # noqa: F401


def test_current_stream_with_and_without_torchs_raw_handle(pkg, monkeypatch):  # noqa: F811
    asked = []

    def current(dev=None):
        asked.append(dev)
        return types.SimpleNamespace(cuda_stream=77)

    monkeypatch.setattr(torch.cuda, "current_stream", current)
    monkeypatch.setattr(pkg, "_raw_stream", lambda dev: 55 + dev)
    assert pkg._stream(None, 3) == 58 and not asked
    monkeypatch.setattr(pkg, "_raw_stream", None)
    assert pkg._stream(None, 3).value == 77 and asked == [3]
    assert pkg._stream(None).value == 77 and asked == [3, None]
    assert pkg._stream(types.SimpleNamespace(cuda_stream=9), 3).value == 9
