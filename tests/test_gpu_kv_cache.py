"""GPU tests of the paged KV cache: dt_kv_write, dt_kv_commit, dt_kv_read.

Codes and scales are defined in fp32 with IEEE operations, so they are compared
exactly with the same operations on the CPU; that the codes are right is
checked against the 64-bit values: a rounding is off by at most half a step,
scale / 2 for int8, |x| 2^-4 (half a step of 3 mantissa bits) or scale 2^-10
(half the smallest step) for e4m3.  The fp32 roundings of X / a, x * (X / a),
a / X and code * scale add at most 4 * 2^-24 of the value each way.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged_attn as oracle
from tests.serving_util import DTYPES, TOP, cuda, page_table, to_codes, values

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import draft_tree_construction_markov_b200 as dt


def _cache(pool, page, hkv, d, code, fill=None):
    c = dt.KVCache.empty(pool, page, hkv, d, DTYPES[code])
    if fill is not None:
        for t in (c.k, c.v):
            t.view(torch.int8).fill_(fill)
        for t in (c.k_scale, c.v_scale):
            if t is not None:
                t.fill_(7.0)
    return c


def _expect(cache, table, page, rows, code):
    """The pool after the rows {(b, position): [Hkv, d]} went in, from its values before."""
    pool = [t.cpu().clone() for t in (cache.k, cache.v)]
    scales = [None if t is None else t.cpu().clone() for t in (cache.k_scale, cache.v_scale)]
    for part in (0, 1):
        for (b, p), x in rows[part].items():
            q, s = to_codes(x, code)
            at = table[b, p // page]
            pool[part][at, :, p % page] = q
            if s is not None:
                scales[part][at, :, p % page] = s
    return pool, scales


def _same(cache, pool, scales):
    bits = lambda t: t.cpu().view(torch.int8 if t.element_size() == 1 else
                                  torch.int16 if t.element_size() == 2 else torch.int32)
    for got, want in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), pool + scales):
        if want is not None:
            assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("code", ["bf16", "f32", "e4m3", "i8"])
@pytest.mark.parametrize("src,d,hkv,page,lens", [
    ("bf16", 128, 8, 16, [1, 0, 37, 5]), ("bf16", 64, 2, 32, [40]), ("f32", 128, 1, 8, [3, 9]),
    ("f32", 64, 3, 128, [130, 1]), ("bf16", 64, 1, 256, [300, 2, 0]), ("bf16", 128, 5, 64, [0, 0])])
def test_write_matches_the_definition(code, src, d, hkv, page, lens):
    g = np.random.default_rng(len(lens) * 100 + d)
    pos = g.integers(0, 50, len(lens))
    table, pool = page_table(g, pos + np.array(lens), page)
    total = sum(lens)
    # slices of one fused tensor: rows further apart than they are long
    fused = torch.randn(max(total, 1), 2 * hkv + 3, d, dtype=DTYPES[src],
                        generator=torch.Generator().manual_seed(d)).mul_(3)[:total]
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cache = _cache(pool, page, hkv, d, code, fill=3)
    rows = [{}, {}]
    for b, n in enumerate(lens):
        for i in range(n):
            for part in (0, 1):
                x = fused[start[b] + i, part * hkv + 1 : part * hkv + 1 + hkv]
                rows[part][b, int(pos[b]) + i] = x.float().numpy()
    want = _expect(cache, table, page, rows, code)
    dev = fused.cuda()
    ws = dt.workspace(dt.kv_workspace_bytes())
    dt.kv_write(dev[:, 1 : 1 + hkv], dev[:, 1 + hkv : 1 + 2 * hkv], cuda(start),
                cuda(pos.astype(np.int32)), cache, cuda(table), ws)
    assert dt.read_status(ws) == 0
    _same(cache, *want)


@pytest.mark.parametrize("code", ["e4m3", "i8"])
def test_codes_are_within_half_a_step_of_the_values(code):
    g = np.random.default_rng(5)
    n, hkv, d, page = 64, 2, 128, 16
    x = (g.standard_normal((n, hkv, d)) * 10.0 ** g.uniform(-30, 30, (n, hkv, 1))).astype(np.float32)
    x[3] = 0.0                      # nothing to scale
    x[4] = 1e-38                    # below 2^-100
    x[5, :, 1:] = 0.0               # one value carries the row
    table, pool = page_table(g, [n], page)
    cache = _cache(pool, page, hkv, d, code)
    ws = dt.workspace(dt.kv_workspace_bytes())
    dx, start, pos = cuda(x), cuda(np.array([0, n], np.int32)), cuda(np.zeros(1, np.int32))
    dt.kv_write(dx, -dx, start, pos, cache, cuda(table), ws)
    k, v = torch.zeros_like(dx), torch.zeros_like(dx)
    dt.kv_read(cache, cuda(table), start, pos, k, v, ws)
    assert dt.read_status(ws) == 0
    x64 = x.astype(np.float64)
    a = np.maximum(np.abs(x64).max(-1, keepdims=True), oracle.TINY)
    step = a / TOP[code]
    half = step / 2 if code == "i8" else np.maximum(np.abs(x64) * 2.0 ** -4, step * 2.0 ** -10)
    bound = half + 8 * 2.0 ** -24 * (np.abs(x64) + half) + 2.0 ** -149
    assert np.all(np.abs(values(k) - x64) <= bound)
    assert torch.equal(k, -v)


@pytest.mark.parametrize("code", ["bf16", "f32", "e4m3", "i8"])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_a_non_finite_row_reads_as_such_and_no_other(code, bad):
    g = np.random.default_rng(2)
    x = g.standard_normal((6, 2, 64)).astype(np.float32)
    x[2, 1, 17] = bad
    table, pool = page_table(g, [6], 8)
    cache = _cache(pool, 8, 2, 64, code)
    ws = dt.workspace(dt.kv_workspace_bytes())
    dx, start, pos = cuda(x), cuda(np.array([0, 6], np.int32)), cuda(np.zeros(1, np.int32))
    dt.kv_write(dx, dx, start, pos, cache, cuda(table), ws)
    k, v = torch.zeros_like(dx), torch.zeros_like(dx)
    dt.kv_read(cache, cuda(table), start, pos, k, v, ws)
    got = k.cpu().numpy()
    hit = np.zeros(x.shape, bool)
    if code in TOP:
        hit[2, 1] = True
        assert np.all(np.isnan(got[hit]))
    else:
        hit[2, 1, 17] = True
        assert np.array_equal(got[hit], x[hit], equal_nan=True)
    assert np.all(np.isfinite(got[~hit]))


@pytest.mark.parametrize("code,out", [("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"),
                                      ("e4m3", "f32"), ("i8", "bf16"), ("i8", "f32"),
                                      ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("d,hkv,page,lens", [(128, 8, 16, [40, 0, 1]), (64, 3, 256, [300, 257])])
def test_read_gathers_code_times_scale_rounded_once(code, out, d, hkv, page, lens):
    g = np.random.default_rng(page)
    first = g.integers(0, 9, len(lens)).astype(np.int32)
    table, pool = page_table(g, first + np.array(lens), page)
    cache = _cache(pool, page, hkv, d, code)
    host = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        q, sc = to_codes(g.standard_normal(t.shape), code)
        t.copy_(q)
        x = q.to(torch.float32)
        if sc is not None:
            s.copy_(sc)
            x = x * sc[..., None]
        host.append(x.to(DTYPES[out]))
    total = sum(lens) + 2  # rows in front of and behind every range stay
    start = (1 + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
    k, v = (torch.full((total, hkv, d), 9.0, dtype=DTYPES[out], device="cuda") for _ in "kv")
    ws = dt.workspace(dt.kv_workspace_bytes())
    dt.kv_read(cache, cuda(table), cuda(start), cuda(first), k, v, ws)
    assert dt.read_status(ws) == 0
    for got, x in ((k, host[0]), (v, host[1])):
        want = torch.full((total, hkv, d), 9.0, dtype=DTYPES[out])
        for b, n in enumerate(lens):
            for i in range(n):
                p = int(first[b]) + i
                want[start[b] + i] = x[table[b, p // page], :, p % page]
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("code", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("batch,nmax,bk", [(1, 1, 1), (5, 32, 7), (3, 64, 16)])
def test_commit_writes_the_root_and_the_accepted_path(code, batch, nmax, bk):
    g = np.random.default_rng(nmax)
    page, hkv, d = 16, 2, 64
    n_acc = g.integers(0, min(bk, nmax) + 1, batch).astype(np.int32)
    n_acc[0] = min(bk, nmax)
    acc = np.full((batch, bk), -1, np.int32)
    for b in range(batch):
        acc[b, : n_acc[b]] = np.sort(g.permutation(nmax)[: n_acc[b]])
    pos = g.integers(0, 100, batch).astype(np.int32)
    table, pool = page_table(g, pos + n_acc + 1, page)
    kt, vt = (torch.randn(batch, nmax + 1, hkv, d, generator=torch.Generator().manual_seed(i)
                          ).to(torch.bfloat16) for i in (1, 2))
    cache = _cache(pool, page, hkv, d, code, fill=5)
    rows = [{}, {}]
    for b in range(batch):
        for i in range(n_acc[b] + 1):
            r = 0 if i == 0 else int(acc[b, i - 1]) + 1
            rows[0][b, int(pos[b]) + i] = kt[b, r].float().numpy()
            rows[1][b, int(pos[b]) + i] = vt[b, r].float().numpy()
    want = _expect(cache, table, page, rows, code)
    ws = dt.workspace(dt.kv_workspace_bytes())
    dt.kv_commit(kt.cuda(), vt.cuda(), cuda(acc), cuda(n_acc), cuda(pos), cache, cuda(table), ws)
    assert dt.read_status(ws) == 0
    _same(cache, *want)


def test_unaligned_source_rows_are_taken_value_by_value():
    g = np.random.default_rng(4)
    table, pool = page_table(g, [5], 8)
    base = torch.randn(5, 1, 67, dtype=torch.float32, generator=torch.Generator().manual_seed(1))
    wide = base.to(torch.bfloat16).cuda()
    src = torch.as_strided(wide, (5, 1, 64), (67, 67, 1), 3)  # rows start on odd elements
    cache, plain = _cache(pool, 8, 1, 64, "e4m3"), _cache(pool, 8, 1, 64, "e4m3")
    ws = dt.workspace(dt.kv_workspace_bytes())
    start, pos = cuda(np.array([0, 5], np.int32)), cuda(np.zeros(1, np.int32))
    dt.kv_write(src, src, start, pos, cache, cuda(table), ws)
    whole = src.contiguous()
    dt.kv_write(whole, whole, start, pos, plain, cuda(table), ws)
    _same(cache, [plain.k.cpu(), plain.v.cpu()], [plain.k_scale.cpu(), plain.v_scale.cpu()])


def test_bad_pages_and_positions_are_dropped_and_recorded():
    """Host-checked bounds first (page table entries and positions are compared before use)."""
    hkv, d, page = 2, 64, 8
    x = torch.randn(12, hkv, d, dtype=torch.bfloat16, device="cuda")
    ws = dt.workspace(dt.kv_workspace_bytes())
    start = cuda(np.array([0, 12], np.int32))
    i32 = lambda *a: cuda(np.array(a, np.int32))
    for table, pos in ((i32(0, 99).view(1, 2), i32(0)), (i32(0, -1).view(1, 2), i32(0)),
                       (i32(0).view(1, 1), i32(0)), (i32(0, 1).view(1, 2), i32(-3))):
        cache = _cache(2, page, hkv, d, "i8", fill=1)
        dt.kv_write(x, x, start, pos, cache, table, ws)
        assert dt.read_status(ws) == 6      # DT_EDEVICE
        assert dt.read_status(ws) == 0      # read once
        good = 8 if int(pos[0]) == 0 else 0
        wrote = (cache.k[0, 0, :, 0].float() != 1).sum() if good else 0
        assert int(wrote) >= good // 2
        out = [torch.full((12, hkv, d), 3.0, device="cuda") for _ in "kv"]
        dt.kv_read(cache, table, start, pos, *out, ws)
        assert dt.read_status(ws) == 6
        if good:
            assert torch.all(out[0][8:] == 0) and torch.all(out[1][8:] == 0)
    acc = i32(5).view(1, 1)                  # a node that the tree has not
    cache = _cache(2, page, hkv, d, "i8", fill=1)
    kt = torch.randn(1, 5, hkv, d, dtype=torch.bfloat16, device="cuda")
    dt.kv_commit(kt, kt, acc, i32(1), i32(0), cache, i32(0, 1).view(1, 2), ws)
    assert dt.read_status(ws) == 6
    assert torch.all(cache.k[0, :, 1] == 1)  # its slot is as it was


def test_write_and_read_replay_in_a_graph_on_another_stream():
    g = np.random.default_rng(9)
    table, pool = page_table(g, [50], 16)
    cache = _cache(pool, 16, 4, 64, "e4m3")
    x = torch.randn(50, 4, 64, dtype=torch.bfloat16, device="cuda")
    out = [torch.zeros_like(x) for _ in "kv"]
    ws = dt.workspace(dt.kv_workspace_bytes())
    args = (cuda(np.array([0, 50], np.int32)), cuda(np.zeros(1, np.int32)))
    dtable = cuda(table)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        dt.kv_write(x, x, *args, cache, dtable, ws)
        dt.kv_read(cache, dtable, *args, *out, ws)
    for seed in (1, 2):
        x.copy_(torch.randn(50, 4, 64, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        q, sc = to_codes(x.float().cpu().numpy(), "e4m3")
        want = (q.float() * sc[..., None]).to(torch.bfloat16)
        assert torch.equal(out[0].cpu(), want) and torch.equal(out[1].cpu(), want)
    assert dt.read_status(ws) == 0
