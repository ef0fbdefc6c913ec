"""Workspaces keep what a captured graph may still write to, within a bound (CPU buffers)."""
import pytest
import torch

import speculative_decoding_fc_gb300 as ds


def _held(ws):
    return sum(b.numel() for b in ws._bufs.values()) + sum(b.numel() for b in ws._outgrown)


def test_slow_growth_holds_a_bounded_total():
    ws = ds.Workspaces()
    for n in range(1000, 200000, 256):
        buf = ws.get("call", "cpu", n)
        assert buf.numel() >= n and buf.dtype is torch.uint8 and not buf.any()
        assert ws.get("call", "cpu", n) is buf and ws.get("call", "cpu", 1) is buf
        # the buffer in use at most twice the need, the outgrown ones together below it
        assert _held(ws) < 4 * n
    assert ws.get("other", "cpu", 100).numel() < 1000


def test_a_large_step_takes_what_it_needs():
    ws = ds.Workspaces()
    assert ws.get("call", "cpu", 1000).numel() == 1000
    assert ws.get("call", "cpu", 50000).numel() == 50000


def test_outgrown_buffers_stay_until_released():
    ws = ds.Workspaces()
    first = ws.get("call", "cpu", 1000)
    first.fill_(7)
    at = first.data_ptr()
    live = ws.get("call", "cpu", 1001)
    del first
    assert [b.data_ptr() for b in ws._outgrown] == [at] and (ws._outgrown[0] == 7).all()
    ws.release()
    assert _held(ws) == live.numel() and ws.get("call", "cpu", 1001) is live


def test_falls_back_to_the_need_when_twice_does_not_fit(monkeypatch):
    ws = ds.Workspaces()
    ws.get("call", "cpu", 1000)
    zeros = torch.zeros

    def limited(n, **kw):
        if n > 1500:
            raise torch.cuda.OutOfMemoryError("no room")
        return zeros(n, **kw)

    monkeypatch.setattr(torch, "zeros", limited)
    assert ws.get("call", "cpu", 1400).numel() == 1400
    with pytest.raises(torch.cuda.OutOfMemoryError):
        ws.get("call", "cpu", 1600)
    assert ws.get("call", "cpu", 1400).numel() == 1400   # still usable
