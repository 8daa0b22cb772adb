"""Which device is current is asked of torch by its public name."""

import contextlib

import torch

from mxfp8_block_scaled_amd import api


def test_public_name(monkeypatch):
    entered = []

    @contextlib.contextmanager
    def device(d):
        entered.append(d.index)
        yield

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    for index, other in ((3, False), (0, True), (7, True)):
        with api._on(torch.device("cuda", index)):
            pass
        assert entered == ([index] if other else [])
        entered.clear()
    with api._on(torch.device("cpu")):
        assert not entered
