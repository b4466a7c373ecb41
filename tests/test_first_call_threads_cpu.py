"""What the binding looks up with its first call is complete for another thread's call
that begins meanwhile."""
import sys

import torch

import reduction_pointwise_row_gb300 as fr


class Watched(dict):
    """A table that notes what another thread would see just before it is filled."""

    def update(self, *a, **kw):
        self.seen = fr._TORCH
        super().update(*a, **kw)


def test_the_dtype_table_is_filled_before_torch_is_published(monkeypatch):
    table = Watched()
    monkeypatch.setattr(fr, "_TORCH", None)
    monkeypatch.setattr(fr, "_LOGIT_DTYPES", table)
    fr._torch()
    assert table.seen is None, "a second thread finds torch there and the table empty"
    assert fr._TORCH is torch and set(table) == {torch.float32, torch.bfloat16}


def test_the_device_lookup_is_there_before_the_stream_lookup(monkeypatch):
    monkeypatch.setattr(fr, "_current_raw_stream", None)
    monkeypatch.setattr(fr, "_current_device", None)
    early = []

    def watch(frame, event, arg):
        if frame.f_code is fr._stream.__code__:
            early.append(fr._current_raw_stream is not None and fr._current_device is None)
            return watch

    sys.settrace(watch)
    try:
        fr._stream()
    except (RuntimeError, AssertionError):
        pass  # no device here
    finally:
        sys.settrace(None)
    assert len(early) > 3 and not any(early), "a second thread finds one lookup without the other"
    assert fr._current_raw_stream is not None and fr._current_device is not None
