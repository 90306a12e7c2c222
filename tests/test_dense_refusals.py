"""What the operators keep between calls, and what they refuse rather than leave out
without a word (CPU where a refusal comes first, GPU where a call has to run)."""

import types

import pytest
import torch

import backward_gate_up_amd as mlp
from backward_gate_up_amd import dense, serve


def test_workspace_sizes_are_kept_by_device(monkeypatch):
    """Two devices with other numbers of compute units need other workspaces: a size
    that one was told is not handed to the other."""
    now = types.SimpleNamespace(device=0)
    asked = []

    def query(*sizes):
        asked.append((now.device, sizes))
        return 1000 * (now.device + 1) + sum(sizes)

    monkeypatch.setattr(serve, "_device", lambda: now.device)
    monkeypatch.setattr(serve, "_L", types.SimpleNamespace(lib=lambda: types.SimpleNamespace(some_workspace_bytes=query)))
    got = []
    for now.device in (0, 1, 0, 1):
        got.append(dense._bytes("some_workspace_bytes", 3, 4))
    assert got == [1007, 2007, 1007, 2007]
    assert asked == [(0, (3, 4)), (1, (3, 4))]  # each asked once
