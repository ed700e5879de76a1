"""Which stream a call takes when it is given none: the current one of the current device, after torch's own
initialisation (which refuses a forked process, for one)."""
import pytest
import torch

import graph_mini_pipeline_amd as gm


class Asked(Exception):
    pass


def test_the_device_is_initialised_first(monkeypatch):
    def lazy():
        raise Asked

    monkeypatch.setattr(torch.cuda, "_lazy_init", lazy)
    with pytest.raises(Asked):
        gm._stream(None)


def test_the_current_stream_of_the_current_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(gm, "_raw_stream", lambda device: 1000 + device)
    assert gm._stream(None).value == 1003


def test_a_torch_without_raw_handles(monkeypatch):
    class Stream:
        cuda_stream = 77

    asked = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    monkeypatch.setattr(gm, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: asked.append(device) or Stream())
    assert gm._stream(None).value == 77 and asked == [2]


def test_a_handle_is_taken_as_it_is():
    assert gm._stream(12345).value == 12345
