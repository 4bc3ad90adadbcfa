"""Arguments of the serving-side calls that no shape or type gives away: where the buffers lie, and
what became of them.  Refused on the host (no GPU needed)."""
import ctypes

import pytest
import torch

import draft_tree_construction_markov_b200 as dt
import draft_tree_construction_markov_b200._lib as L
from tests.test_serving_host import _attn, _commit, _logits, _read, _tree, _write

EINVAL, EWORKSPACE = L.DT_EINVAL, L.DT_EWORKSPACE
CALLS = [_write, _commit, _read, _attn, _tree, _logits]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("at", [0x1001, 0x1004, 0x1008, 0x100c])
def test_a_workspace_off_16_bytes_is_refused(call, at):
    """Behind its header lie records that are read and written 16 bytes at a time."""
    assert call(ws=ctypes.c_void_p(at)) == EINVAL
    assert call(ws=ctypes.c_void_p(at), bytes=8) == EWORKSPACE
