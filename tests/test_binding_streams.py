"""How the binding's functions take `stream`, without a GPU: by name or by position, entered only if it is not
the current one."""
import contextlib
import inspect
import types

import pytest

from combine_warp_top_router_b200 import binding


def test_stream_is_the_last_parameter_everywhere():
    taking = [f for n, f in vars(binding).items()
              if n.startswith("md_") and inspect.isfunction(f) and "stream" in inspect.signature(f).parameters]
    assert len(taking) >= 24
    for f in taking:
        assert list(inspect.signature(f).parameters)[-1] == "stream"
        assert hasattr(f, "__wrapped__"), f.__name__  # allocates as its stream's


@pytest.mark.parametrize("current", [7, 8])
@pytest.mark.parametrize("by", ["name", "position", "neither"])
def test_stream_by_name_and_by_position(monkeypatch, current, by):
    entered = []

    @contextlib.contextmanager
    def enter(s):
        entered.append(s)
        yield

    monkeypatch.setattr(binding, "_raw_stream", lambda device: current)
    monkeypatch.setattr(binding.torch.cuda, "stream", enter)

    @binding._on_its_stream
    def f(x, out=None, dev_status=None, stream=None):
        return x, out, dev_status, stream

    s = types.SimpleNamespace(device_index=0, cuda_stream=8)
    if by == "neither":
        assert f(1) == (1, None, None, None) and f(1, 2, dev_status=3) == (1, 2, 3, None) and f(1, 2, 3, None)[3] is None
        assert entered == []
        return
    got = f(1, dev_status=3, stream=s) if by == "name" else f(1, None, 3, s)
    assert got == (1, None, 3, s)
    assert entered == ([] if current == 8 else [s])
    with pytest.raises(TypeError):
        f(1, 2, 3, s, 5)
    with pytest.raises(TypeError):
        f(1, 2, 3, s, stream=s)
