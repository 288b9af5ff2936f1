"""The binding of the linear attention and the norm, without a GPU."""
import types

import torch

from gated_delta_rule_108_b200 import kda


def test_the_current_stream_without_torchs_private_call(monkeypatch):
    """Another torch may lack it: the public call serves."""
    monkeypatch.setattr(kda.torch, "_C", types.SimpleNamespace())
    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: asked.append(i) or types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(kda, "_current_raw", kda._current_raw_stream())
    assert kda._raw_stream(None, types.SimpleNamespace(index=3)) == 77 and asked == [3]
    assert kda._raw_stream(types.SimpleNamespace(cuda_stream=5), None) == 5
