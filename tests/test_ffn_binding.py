"""The feed-forward operators' binding on the CPU: what it does before a call
reaches the library."""
from __future__ import annotations

import torch

import hyper_connection_rank_amd as hc


def test_a_workspace_of_the_call_s_own_has_only_its_counters_cleared(monkeypatch):
    """The counters have to be zero; clearing the rest would write up to hundreds of megabytes a call."""
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(0xA5))
    ws = hc.ffn._scratch(None, 1 << 20, torch.device("cpu"))
    assert ws.numel() == 1 << 20 and ws.dtype == torch.uint8
    assert not ws[:4096].any()
    assert (ws[4096:] == 0xA5).all()
