"""The binding's cached workspace and graph capture (no GPU needed: torch's
stream, capture and allocation calls are replaced by stand-ins).

A captured graph keeps the addresses its kernels were given, and no reference
to a tensor.  A workspace from the cache could then be replaced by a larger
one, and its memory be another tensor's, while the graph still writes there;
and graphs captured on one stream would share it whatever streams they are
replayed on."""
import types

import pytest
import torch

from deformable_convolution_amd import dc1d, sequence


@pytest.fixture
def fake(monkeypatch):
    state = types.SimpleNamespace(capturing=False, stream=7)
    empty = torch.empty
    monkeypatch.setattr(dc1d, "_ws_cache", {})
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=state.stream))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw))
    return state


def both():
    """How the two bindings ask for one."""
    device = torch.device("cuda", 0)
    return [lambda n: dc1d._workspace(n, device), lambda n: sequence._get(n, 0)]


@pytest.mark.parametrize("get", both())
def test_a_captured_call_does_not_take_the_cached_workspace(fake, get):
    eager = get(4096)
    assert get(1000) is eager
    fake.capturing = True
    first, second = get(1000), get(1000)
    assert len({t.data_ptr() for t in (eager, first, second)}) == 3
    assert first.numel() >= 1000 and second.numel() >= 1000
    fake.capturing = False
    assert get(1000) is eager


@pytest.mark.parametrize("get", both())
def test_a_captured_call_leaves_nothing_in_the_cache(fake, get):
    # what it allocates belongs to the graph's pool, and goes with the graph
    fake.capturing = True
    captured = get(4096)
    fake.capturing = False
    assert dc1d._ws_cache == {}
    assert get(4096).data_ptr() != captured.data_ptr()
