"""Where a call's stream comes from: torch's public functions alone."""
import os
import re

import torch

from io_aware_exact_21_b200 import binding as bd


class Fake:
    cuda_stream = 0x1234
    native_handle = 0x5678


def test_the_current_stream_is_the_public_one(monkeypatch):
    # of the current device
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.accelerator, "current_stream", lambda device=None: Fake() if device == 3 else None)
    assert bd._stream(None) == 0x5678


def test_a_given_stream():
    assert bd._stream(0) == 0 and bd._stream(7) == 7 and bd._stream(Fake()) == 0x1234


def test_no_private_torch_names():
    with open(os.path.join(os.path.dirname(bd.__file__), "binding.py")) as f:
        assert not re.findall(r"torch\._\w+|\._C\b", f.read())
