"""Where a call's stream comes from: torch's public functions alone."""
import os
import re

import torch

from io_aware_exact_21_b200 import binding as bd


class Fake:
    cuda_stream = 0x1234


def test_the_current_stream_is_the_public_one(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Fake())
    assert bd._stream(None) == 0x1234


def test_a_given_stream():
    assert bd._stream(0) == 0 and bd._stream(7) == 7 and bd._stream(Fake()) == 0x1234


def test_no_private_torch_names():
    with open(os.path.join(os.path.dirname(bd.__file__), "binding.py")) as f:
        assert not re.findall(r"torch\._\w+|\._C\b", f.read())
