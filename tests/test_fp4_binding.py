"""Memory that the 4-bit operators' torch binding takes itself (no GPU: calls of the library are recorded)."""
from __future__ import annotations

import contextlib

import pytest

import expert_ffn_gb300 as mx


class Handle:
    """A stream of another library: its handle alone."""

    cuda_stream = 0x1234560


@pytest.mark.parametrize("stream,taken_on", [(None, None), (0, "default 0"), (0x1234560, 0x1234560), (Handle, 0x1234560)])
def test_scales_are_packed_into_memory_of_the_stream_that_packs_them(monkeypatch, stream, taken_on):
    """Of the current stream's pool the block may still be in use by that stream's earlier work."""
    import torch

    class OnDevice(torch.Tensor):
        def get_device(self):
            return 0

    current, taken, calls = [None], [], []

    @contextlib.contextmanager
    def stream_context(s):
        before, current[0] = current[0], s
        yield
        current[0] = before

    empty = torch.empty

    def record_empty(*a, **kw):
        taken.append(current[0])
        return empty(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: f"default {device}")
    monkeypatch.setattr(torch, "empty", record_empty)
    mx._torch()
    monkeypatch.setattr(mx, "_on", lambda dev, fn, *args: calls.append((dev, args)))
    monkeypatch.setattr(mx._t, "stream", lambda dev: 77)
    w = torch.zeros(64, 128, dtype=torch.uint8).as_subclass(OnDevice)
    scales = torch.zeros(64, 16, dtype=torch.uint8).view(torch.float8_e4m3fn).as_subclass(OnDevice)
    weight = mx.Fp4Weight(w, scales, stream=stream)
    assert taken == [taken_on]
    (dev, args), = calls
    assert dev == 0 and weight.packed.data_ptr() in args
    assert args[-1] == (77 if stream is None else 0 if stream == 0 else 0x1234560)
