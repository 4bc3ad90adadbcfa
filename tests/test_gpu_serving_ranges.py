"""GPU tests of ranges: prompt lengths and lists of the logits processing that do not fit, and which
request of many a row of the cache belongs to.  Compared on the device before any use."""
import numpy as np
import pytest
import torch

from tests.serving_util import DTYPES, cuda, page_table, to_codes

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


# --------------------------------------------------- rows of many requests --
def _lens(g, batch, kind):
    """Rows a request: some of none at the front, in runs and at the end."""
    n = g.integers(1, 4, batch)
    if kind == "gaps":
        n[: batch // 5] = 0
        n[-(batch // 7) - 1 :] = 0
        n[batch // 3 : batch // 2] = 0
        n[batch // 2] = 5
    elif kind == "one":
        n[:] = 0
        n[g.integers(0, batch)] = 3
    return n


@pytest.mark.parametrize("kind", ["all", "gaps", "one"])
@pytest.mark.parametrize("batch", [31, 32, 33, 64, 65, 333, 1024])
def test_rows_of_many_requests_go_to_their_own_pages(batch, kind):
    g = np.random.default_rng(batch)
    page, hkv, d, lead = 8, 1, 64, 3
    n = _lens(g, batch, kind)
    pos = g.integers(0, 12, batch)
    table, pool = page_table(g, pos + n, page)
    start = (lead + np.concatenate([[0], np.cumsum(n)])).astype(np.int32)   # row_start[0] > 0
    total = int(start[-1]) + 2
    x = torch.randn(total, hkv, d, generator=torch.Generator().manual_seed(batch)).to(torch.bfloat16)
    q, s = to_codes(x.float().numpy(), "i8")
    cache = dt.KVCache.empty(pool, page, hkv, d, DTYPES["i8"])
    want, want_s = torch.zeros_like(cache.k, device="cpu"), torch.zeros_like(cache.k_scale, device="cpu")
    back = torch.full((total, hkv, d), 9.0)
    for b in range(batch):
        for i in range(n[b]):
            p, r = int(pos[b]) + i, start[b] + i
            want[table[b, p // page], :, p % page] = q[r]
            want_s[table[b, p // page], :, p % page] = s[r]
            back[r] = q[r].float() * s[r][..., None]
    ws, dx = dt.workspace(dt.kv_workspace_bytes()), x.cuda()
    where = (_i32(start), _i32(pos))
    dt.kv_write(dx, -dx, *where, cache, cuda(table), ws)
    assert dt.read_status(ws) == 0
    assert torch.equal(cache.k.cpu(), want) and torch.equal(cache.v.cpu(), -want)
    assert torch.equal(cache.k_scale.cpu(), want_s) and torch.equal(cache.v_scale.cpu(), want_s)
    k, v = (torch.full((total, hkv, d), 9.0, device="cuda") for _ in "kv")
    dt.kv_read(cache, cuda(table), *where, k, v, ws)
    assert dt.read_status(ws) == 0
    assert torch.equal(k.cpu(), back)
    assert torch.equal(v.cpu()[lead : start[-1]], -back[lead : start[-1]])
    assert torch.all(v[:lead] == 9) and torch.all(v[int(start[-1]) :] == 9)
