"""First calls of several threads (host-side): what a call takes from torch is in place before torch itself, which
says that it is, is published."""
import torch

from cnn_convolution_implicit_gb300 import rows


def test_torch_is_published_last(monkeypatch):
    for name in ("_t", "_empty", "_empty_like", "_bf16", "_f32"):
        monkeypatch.setattr(rows, name, None)
    seen = []

    class Watched:
        def __getattr__(self, name):  # another thread may run at each of these points
            seen.append(rows._t is None or None not in (rows._empty, rows._empty_like, rows._bf16, rows._f32))
            return getattr(torch, name)

    watched = Watched()
    monkeypatch.setattr(rows, "_torch", lambda: watched)
    assert rows._start() is watched and rows._t is watched
    assert seen and all(seen)
    assert rows._empty is torch.empty and rows._empty_like is torch.empty_like
    assert rows._bf16 is torch.bfloat16 and rows._f32 is torch.float32
