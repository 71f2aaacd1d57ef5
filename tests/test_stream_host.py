"""How the binding finds the current stream, on torch builds with and without
the calls that return its address directly."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def ga():
    import gradient_aggregation_amd as ga
    return ga


def stand_in(**calls):
    stream = types.SimpleNamespace(cuda_stream=77)
    return types.SimpleNamespace(_C=types.SimpleNamespace(**calls),
                                 cuda=types.SimpleNamespace(current_stream=lambda: stream))


def test_with_the_direct_calls(ga, monkeypatch):
    t = stand_in(_cuda_getDevice=lambda: 3, _cuda_getCurrentRawStream=lambda device: 100 + device)
    monkeypatch.setattr(ga, "_torch", lambda: t)
    assert ga._stream_ptr() == 103


@pytest.mark.parametrize("calls", [{}, {"_cuda_getDevice": lambda: 0}, {"_cuda_getCurrentRawStream": lambda device: 1}])
def test_without_them(ga, monkeypatch, calls):
    t = stand_in(**calls)
    monkeypatch.setattr(ga, "_torch", lambda: t)
    assert ga._stream_ptr() == 77
