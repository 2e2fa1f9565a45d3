"""The stream that the binding passes on, with and without torch's short way to it."""
import types

import pytest

kvq = pytest.importorskip("int4_quantized_paged_gb300.kvq",
                          reason="libkvq.so not built (run __graft_entry__.build())")


def test_the_current_stream_of_the_current_device(monkeypatch):
    monkeypatch.setattr(kvq, "_device", lambda: 3, raising=False)
    monkeypatch.setattr(kvq, "_raw_stream", lambda device: 1000 + device, raising=False)
    assert kvq._stream(None) == 1003


@pytest.mark.parametrize("missing", ["_device", "_raw_stream"])
def test_a_torch_without_the_short_way(monkeypatch, missing):
    monkeypatch.setattr(kvq, missing, None, raising=False)
    monkeypatch.setattr(kvq.torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert kvq._stream(None) == 77


def test_a_given_stream_is_taken_as_it_is():
    assert kvq._stream(5) == 5 and kvq._stream(0) == 0
    assert kvq._stream(types.SimpleNamespace(cuda_stream=9)) == 9
