"""A workspace that a call makes for itself belongs to the stream it launches on."""
import contextlib
import types

import pytest
import torch

from decode_attention_paged_pa_gb300 import binding


class Seen:
    """Stands in for torch.cuda: streams are what is entered, allocations what is made in them."""

    def __init__(self, monkeypatch, current=3):
        self.inside, self.made = [], []
        monkeypatch.setattr(binding, "_raw_stream", lambda device: current)
        monkeypatch.setattr(binding.torch.cuda, "stream", self.enter)
        monkeypatch.setattr(binding.torch.cuda, "ExternalStream", lambda handle, device: ("external", handle, device))
        monkeypatch.setattr(binding.torch, "empty", self.empty)

    @contextlib.contextmanager
    def enter(self, stream):
        self.inside.append(stream)
        yield
        self.inside.pop()

    def empty(self, n, dtype, device):
        self.made.append((n, list(self.inside)))
        return "workspace"


def test_on_the_current_stream(monkeypatch):
    seen = Seen(monkeypatch)
    for stream in (None, 3, types.SimpleNamespace(cuda_stream=3)):
        assert binding._new_workspace(1000, 0, stream) == "workspace"
    assert seen.made == [(1000, [])] * 3


@pytest.mark.parametrize("stream,handle", [(0, 0), (1, 0), (2, 2), (1 << 40, 1 << 40),
                                           (types.SimpleNamespace(cuda_stream=48), 48)])
def test_on_another_stream(monkeypatch, stream, handle):
    seen = Seen(monkeypatch)
    binding._new_workspace(10, 0, stream)
    assert seen.made == [(256, [("external", handle, torch.device("cuda", 0))])]


def test_no_entry_point_makes_one_otherwise():
    import inspect

    for name, fn in inspect.getmembers(binding, inspect.isfunction):
        if name != "_new_workspace":
            assert "torch.empty" not in inspect.getsource(fn), name
