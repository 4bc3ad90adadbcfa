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


def _cpu_cache(dtype=torch.int8):
    return dt.KVCache.empty(4, 16, 2, 64, dtype, device="cpu")


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "n_pages", "Hkv", "page_size", "d", "device"])
def test_a_cache_s_attributes_cannot_be_set(name):
    """The calls go by what the constructor saw: a larger pool assigned later would leave them on the
    old one, which nothing keeps alive."""
    c = _cpu_cache()
    old = getattr(c, name)
    with pytest.raises(AttributeError):
        setattr(c, name, torch.zeros(8, 2, 16, 64, dtype=torch.int8))
    assert getattr(c, name) is old
    c.k[0].fill_(3)                                       # filling them is what they are for


@pytest.mark.parametrize("dtype,part", [(torch.bfloat16, 0), (torch.bfloat16, 1), (torch.int8, 0), (torch.int8, 1),
                                        (torch.int8, 2), (torch.int8, 3)])
@pytest.mark.parametrize("grow", [False, True])
def test_a_cache_whose_storage_has_moved_is_refused(dtype, part, grow):
    c = _cpu_cache(dtype)
    t = (c.k, c.v, c.k_scale, c.v_scale)[part]
    if grow:
        t.resize_(64, *t.shape[1:])
    else:
        t.data = torch.zeros_like(t)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    x, q = torch.zeros(10, 2, 64), torch.zeros(10, 4, 64, dtype=torch.bfloat16)
    tree, kt = torch.zeros(2, 9, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 9, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: dt.kv_write(x, x, i(3), i(2), c, i(2, 4), ws),
                 lambda: dt.kv_read(c, i(2, 4), i(3), i(2), x, x.clone(), ws),
                 lambda: dt.kv_commit(kt, kt, i(2, 4), i(2), i(2), c, i(2, 4), ws),
                 lambda: dt.paged_attn(q, i(3), c, i(2, 4), i(2), 0.1, q.clone(), ws, max_rows=5),
                 lambda: dt.tree_verify_attn_paged(tree, c, i(2, 4), i(2), kt, kt,
                                                   torch.zeros(2, 8, dtype=torch.int64), i(2), 0.1, tree.clone(),
                                                   ws)):
        with pytest.raises(ValueError, match="moved"):
            call()


def at(x):
    return ctypes.c_void_p(0x100000 + x)


def _answers(call, code, **kw):
    """EINVAL where code says so; else the arguments are fine, and without a device the launch fails.
    With one it would run on addresses that are none: such a call is not made."""
    if code:
        assert call(**kw) == code
    elif not torch.cuda.is_available():
        assert call(**kw) == L.DT_ECUDA


# 10 rows of 4 heads of 64 bf16: 512 bytes a row
@pytest.mark.parametrize("out,ld,code", [
    (0, 256, EINVAL), (16, 256, EINVAL), (-16, 256, EINVAL), (5119 // 16 * 16, 256, EINVAL),
    (-5120 + 16, 256, EINVAL), (5120, 256, None), (-5120, 256, None),
    # rows of a fused projection, 8192 bytes apart: the output may lie between two of them
    (512, 4096, None), (8192 - 5120, 4096, None), (8192 - 5120 + 16, 4096, EINVAL), (496, 4096, EINVAL),
    (9 * 8192 + 512, 4096, None), (9 * 8192 + 496, 4096, EINVAL)])
def test_an_output_over_the_queries_is_refused(out, ld, code):
    """Rows that are done again read their query after outputs were written."""
    _answers(_attn, code, q=at(0), out=at(out), ld=ld)


# 18 rows: q 4 heads of 64 bf16 (9216 bytes), tree rows 2 heads (4608 bytes)
@pytest.mark.parametrize("name,size", [("q", 9216), ("k", 4608), ("v", 4608)])
def test_an_output_over_what_a_tree_call_reads_is_refused(name, size):
    far = dict(q=at(1 << 20), k=at(2 << 20), v=at(3 << 20))
    for x, code in ((0, EINVAL), (size - 16, EINVAL), (16 - 9216, EINVAL), (size, None), (-9216, None)):
        _answers(_tree, code, **{**far, name: at(0)}, out=at(x))


@pytest.mark.parametrize("dtype,out", [(L.DT_F32, 10 * 1024 - 16), (L.DT_BF16, 10 * 512 - 16)])
def test_the_overlap_goes_by_the_type(dtype, out):
    _answers(_attn, EINVAL, q=at(0), out=at(out), ld=256, dt=dtype)
    _answers(_attn, None, q=at(0), out=at(out + 16), ld=256, dt=dtype)


def test_a_workspace_holds_what_its_call_can_leave_and_no_more():
    """Two partials of (sums, maximum and sum of weights) a pair, for every worker: 296 blocks of row
    tiles, or 148 blocks of 11 workers of at most 16 pairs, which trees never have; and 32 bytes of
    records a worker, with the header and paddings below a kilobyte."""
    part = lambda workers, pairs, d: workers * (2 * pairs * (4 * d + 8) + 32)
    for d in (64, 128):
        for rows, pairs in ((4, 16), (1, 4), (33, 132), (65, 260)):
            tiles, few = part(296, min(pairs, 128), d), part(148 * 11, min(pairs, 16), d)
            assert 0 <= dt.paged_attn_workspace_bytes(1, rows, 32, 8, d) - max(tiles, few) < 1024
            if rows > 1:
                assert 0 <= dt.verify_paged_workspace_bytes(1, rows - 1, 32, 8, d) - tiles < 1024


def test_lists_of_logits_that_do_not_belong_together_are_refused():
    z, ws = torch.zeros(2, 1, 50), torch.zeros(256, dtype=torch.uint8)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for bad in (dict(bias_value=torch.zeros(3)), dict(bias_token=i(2), bias_value=torch.zeros(3), bias_start=i(3)),
                dict(bias_token=i(0), bias_value=torch.zeros(3), bias_start=i(3)),
                dict(history=i(0), history_start=i(2)), dict(mask=i(0, 2), mask_row=i(2))):
        with pytest.raises(ValueError):
            dt.logits_process(z, torch.zeros_like(z), ws, **bad)
