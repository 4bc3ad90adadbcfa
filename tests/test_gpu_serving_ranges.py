"""GPU tests of ranges that do not fit, in the lists of the logits processing.  Compared on the device
before any use."""
import numpy as np
import pytest
import torch

from tests.serving_util import cuda

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import draft_tree_construction_markov_b200 as dt

EDEVICE = 6


def _i32(a):
    return cuda(np.asarray(a, np.int32))


def _f32(*a):
    return cuda(np.asarray(a, np.float32))


@pytest.mark.parametrize("n_prompt,as_if,status", [(0, 0, 0), (2, 2, 0), (3, 3, 0), (4, 3, EDEVICE), (-1, 0, EDEVICE),
                                                   (2 ** 31 - 1, 3, EDEVICE), (-2 ** 31, 0, EDEVICE)])
def test_a_prompt_length_outside_its_history_is_recorded_and_clamped(n_prompt, as_if, status):
    x = torch.ones(2, 1, 40, device="cuda")
    out, ws = torch.zeros_like(x), dt.workspace(dt.logits_workspace_bytes())
    dt.logits_process(x, out, ws, history=_i32([9, 7, 8, 5]), history_start=_i32([0, 1, 4]),
                      n_prompt=_i32([1, n_prompt]), frequency=_f32(0.25, 0.25), repetition=_f32(2, 2))
    assert dt.read_status(ws) == status
    want = x.clone()
    want[0, 0, 9] = 0.5                      # the prompt's tokens are divided, the others counted too
    for i, t in enumerate((7, 8, 5)):
        want[1, 0, t] = 0.5 if i < as_if else 0.25
    assert torch.equal(out, want)


def _empty(dtype=torch.int32, *more):
    return torch.empty(0, *more, dtype=dtype, device="cuda")


@pytest.mark.parametrize("args,status", [
    (dict(history=lambda: _empty(), history_start=lambda: _i32([0, 0, 0])), 0),
    (dict(history=lambda: _empty(), history_start=lambda: _i32([0, 0, 2])), EDEVICE),
    (dict(history=lambda: _empty(), history_start=lambda: _i32([0, 0, 0]), n_prompt=lambda: _i32([0, 3])), EDEVICE),
    (dict(history=lambda: _empty(), history_start=lambda: None, n_prompt=lambda: _i32([0, 3])), 0),
    (dict(bias_token=lambda: _empty(), bias_value=lambda: _empty(torch.float32), bias_start=lambda: _i32([0, 0, 0])), 0),
    (dict(bias_token=lambda: _empty(), bias_value=lambda: _empty(torch.float32), bias_start=lambda: _i32([0, 1, 1])),
     EDEVICE),
    (dict(mask=lambda: _empty(torch.int32, 2)), 0),
    (dict(mask=lambda: _empty(torch.int32, 2), mask_row=lambda: _i32([[-1], [-1]])), 0),
    (dict(mask=lambda: _empty(torch.int32, 2), mask_row=lambda: _i32([[-1], [0]])), EDEVICE)])
def test_what_points_into_an_empty_list_is_read(args, status):
    x = torch.randn(2, 1, 40, device="cuda")
    out, ws = torch.zeros_like(x), dt.workspace(dt.logits_workspace_bytes())
    dt.logits_process(x, out, ws, repetition=_f32(2, 2), **{k: f() for k, f in args.items()})
    assert dt.read_status(ws) == status
    assert torch.equal(out, x)
