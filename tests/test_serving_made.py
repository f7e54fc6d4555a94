"""Which stream a call makes its own tensors on (CPU only: torch's stream
functions are replaced by records of their calls)."""
import contextlib

import pytest


class Like:
    device = "cuda:0"

    def get_device(self):
        return 0


@pytest.mark.parametrize("given,current,want", [
    (None, 0, None), (0, 0, None), (7, 7, None),           # already current
    (0, 7, "default"), (1, 7, "default"), (8, 7, 8), (8, 0, 8)])
def test_stream_of_made_tensors(given, current, want, monkeypatch):
    import torch
    import token_level_dynamic_b200 as w
    entered = []

    @contextlib.contextmanager
    def stream(s):
        entered.append(s)
        yield

    monkeypatch.setattr(w, "_raw_stream", lambda dev: current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: "default")
    monkeypatch.setattr(torch.cuda, "stream", stream)
    made = w._made(lambda shape, dtype, device: (shape, dtype, device), (3,), "dtype", Like(), given)
    assert made == ((3,), "dtype", "cuda:0")
    assert entered == ([] if want is None else [want])
