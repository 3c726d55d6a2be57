"""Which device and stream a binding call makes current, decided without a GPU."""
import inspect
import re

import pytest
import torch

from w8a8_int8_quantized_norm_b200 import sq


class _Stream:
    def __init__(self, device):
        self.device = torch.device(device)


def test_scope_makes_the_tensors_device_current(monkeypatch):
    monkeypatch.setattr(sq, "_raw_device", lambda: 0)
    other = sq._scope(torch.device("cuda", 1), None)
    assert isinstance(other, torch.cuda.device) and other.idx == 1
    assert sq._scope(torch.device("cuda", 0), None) is sq._NO_SCOPE
    assert sq._scope(torch.device("cpu"), None) is sq._NO_SCOPE


def test_scope_refuses_a_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(sq, "_raw_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        sq._scope(torch.device("cuda", 1), _Stream("cuda:0"))


def test_every_call_that_takes_a_stream_allocates_in_its_scope():
    """In the source of each call, allocations and the library call stand inside the scope."""
    checked = 0
    for name, fn in inspect.getmembers(sq, inspect.isfunction):
        if "stream" not in inspect.signature(fn).parameters or name in ("_scope", "_stream",
                                                                       "get_device_error"):
            continue
        body = inspect.getsource(fn)
        if "_scope(" not in body:  # hands the stream on to a call that opens it
            assert not re.search(r"torch\.(empty|zeros)\(|_check\(", body), name
            continue
        before = body[:body.index("with _scope(")]
        assert not re.search(r"torch\.(empty|zeros)\(|_check\(", before), name
        checked += 1
    assert checked >= 25
