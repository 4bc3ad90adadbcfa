"""GPU tests of dt_paged_attn and dt_tree_verify_attn_paged against fp64.

Error bound of an output o = sum w_j v_j / sum w_j, with A = sum w_j |v_j| / sum w_j:
  - bf16: o rounded once (2^-8 |o|), every weight rounded to bf16 before the
    second product (2^-8 A), as the header says;
  - fp32: no such rounding;
  - scores: a sum of d products and the scales, each within 2^-24 of the sum of
    magnitudes B = scale * sum |q k|: ds = (d + 8) 2^-24 B, and a weight moves
    by exp(ds), numerator and denominator: 2 ds A;
  - sums over keys in fp32: L 2^-24 A each for numerator and denominator, and
    the exponential's own error (2^-21).
"""
import numpy as np
import pytest
import torch

from oracle import paged_attn as oracle
from tests.serving_util import DTYPES, cuda, page_table, random_tree, to_codes, values

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import draft_tree_construction_markov_b200 as dt


def _bound(o, mag, big, d, keys, kind):
    ds = (d + 8) * 2.0 ** -24 * big[..., None]
    rel = 2 * ds + (2 * keys * 2.0 ** -24 + 2.0 ** -20)
    tol = rel * mag + 2.0 ** -24 * np.abs(o)
    if kind == "bf16":
        tol = tol + 2.0 ** -8 * mag * (1 + rel) + 2.0 ** -8 * (np.abs(o) + tol + 2.0 ** -8 * mag)
    return tol + 2.0 ** -126


class Pool:
    """A cache of random rows on the GPU and its fp64 values."""

    def __init__(self, g, lens, page, hkv, d, code, poison=False):
        self.table, n = page_table(g, lens, page)
        self.cache = dt.KVCache.empty(n, page, hkv, d, DTYPES[code])
        self.host = []
        for t, s in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            q, sc = to_codes(g.standard_normal(t.shape), code)
            if poison:
                # slots that hold no request's position are not numbers
                used = torch.zeros(t.shape[0], t.shape[2], dtype=torch.bool)
                for b, L in enumerate(lens):
                    for p in range(L):
                        used[self.table[b, p // page], p % page] = True
                hole = ~used[:, None].expand(t.shape[:3])
                if sc is not None:
                    sc = torch.where(hole, torch.nan, sc)
                if code in ("bf16", "f32"):
                    q = torch.where(hole[..., None], torch.nan, q.float()).to(q.dtype)
                elif code == "e4m3":
                    q.view(torch.uint8)[hole] = 0x7F
            t.copy_(q)
            if sc is not None:
                s.copy_(sc)
            self.host.append((values(q), None if sc is None else values(sc)))

    def rows(self, b, length):
        return [oracle.gather(x, s, self.table[b], length) for x, s in self.host]


def _q(g, shape, kind):
    t = torch.as_tensor(g.standard_normal(shape).astype(np.float32)).to(DTYPES[kind])
    return t.cuda(), values(t)


def _chunk(g, lens, rows, page, hq, hkv, d, code, kind, window=0, sink=0, poison=False, max_rows=None,
           strided=False):
    pool = Pool(g, lens, page, hkv, d, code, poison)
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    total = int(start[-1])
    q, q64 = _q(g, (total + 2, hq + (3 if strided else 0), d), kind)
    q, q64 = q[1:-1, :hq], q64[1:-1, :hq]
    out = torch.full((total, hq, d), 7.0, dtype=DTYPES[kind], device="cuda")
    ws = dt.workspace(dt.paged_attn_workspace_bytes(len(lens), total, hq, hkv, d))
    scale = d ** -0.5
    dt.paged_attn(q, cuda(start), pool.cache, cuda(pool.table), cuda(np.array(lens, np.int32)), scale,
                  out, ws, max_rows=max_rows or max(max(rows), 1), window=window, n_sink=sink)
    assert dt.read_status(ws) == 0
    got = values(out)
    worst = 0.0
    for b, L in enumerate(lens):
        if rows[b] == 0:
            continue
        k, v = pool.rows(b, L)
        qb = q64[start[b] : start[b + 1]]
        # long chunks: some of the rows, the first and the last among them
        n = rows[b]
        pick = np.arange(n) if n * hq * L < 3e6 else np.unique(
            np.concatenate([[0, 1, n - 1], g.integers(0, n, 12)]))
        ok = np.stack([oracle.seen_positions(L - n + i, L, window, sink) for i in pick])
        o, mag, big = oracle.attend(qb[pick], k, v, ok, scale)
        tol = _bound(o, mag, big, d, L, kind)
        err = np.abs(got[start[b] : start[b + 1]][pick] - o)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        worst = max(worst, float((err / tol).max()))
    return worst


SHAPES = [  # lens, rows, page, Hq, Hkv, d
    ([1], [1], 16, 2, 2, 64),
    ([33, 1, 200], [1, 1, 1], 16, 32, 8, 128),
    ([129, 128, 127, 17], [1, 1, 1, 1], 128, 8, 1, 64),
    ([700, 64], [2, 4], 64, 12, 4, 128),
    ([300, 5, 40], [64, 5, 0], 32, 8, 2, 64),
    ([1000], [257], 8, 6, 2, 128),
    ([513, 140], [130, 140], 256, 4, 4, 128),
    ([90, 600, 31], [7, 1, 31], 16, 10, 2, 64),
    ([70], [33], 64, 33, 1, 128),
]


@pytest.mark.parametrize("code", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_chunk_bf16(code, shape):
    _chunk(np.random.default_rng(len(shape[0]) + shape[2]), *shape, code, "bf16")


@pytest.mark.parametrize("code", ["f32", "bf16", "e4m3", "i8"])
@pytest.mark.parametrize("shape", SHAPES[:5])
def test_chunk_f32(code, shape):
    _chunk(np.random.default_rng(3), *shape, code, "f32")


@pytest.mark.parametrize("code,kind", [("bf16", "bf16"), ("i8", "bf16"), ("e4m3", "f32")])
@pytest.mark.parametrize("window,sink", [(1, 0), (7, 0), (64, 4), (128, 1), (200, 17), (10000, 4),
                                         (50, 10000)])
@pytest.mark.parametrize("shape", [([500, 33, 210], [1, 1, 1], 16, 8, 2, 64),
                                   ([700, 130], [300, 130], 64, 8, 2, 128)])
def test_window_and_first_tokens(code, kind, window, sink, shape):
    _chunk(np.random.default_rng(window), *shape, code, kind, window, sink)


@pytest.mark.parametrize("code", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("rows", [[1, 1, 1], [20, 33, 64]])
def test_what_no_row_sees_may_be_anything(code, rows):
    """Slots behind a request's last position, unused pages: NaN, and page -1."""
    _chunk(np.random.default_rng(1), [50, 33, 200], rows, 32, 8, 2, 128, code, "bf16", poison=True)
    _chunk(np.random.default_rng(1), [50, 33, 200], rows, 32, 8, 2, 128, code, "bf16", 20, 3,
           poison=True)


@pytest.mark.parametrize("code", ["bf16", "i8"])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_pages_behind_the_window_are_not_read(code, n):
    g = np.random.default_rng(n)
    L, page, window, sink = 1000, 16, 100, 5
    pool = Pool(g, [L], page, 2, 64, code)
    q, q64 = _q(g, (n, 4, 64), "bf16")
    out = torch.zeros_like(q)
    ws = dt.workspace(dt.paged_attn_workspace_bytes(1, n, 4, 2, 64))
    k, v = pool.rows(0, L)
    o, mag, big = oracle.chunk(q64, k, v, L, window, sink, 0.125)
    first = L - n - window + 1
    pool.table[0, 1 : first // page] = -1          # freed: no row sees them
    dt.paged_attn(q, cuda(np.array([0, n], np.int32)), pool.cache, cuda(pool.table),
                  cuda(np.array([L], np.int32)), 0.125, out, ws, max_rows=n, window=window, n_sink=sink)
    assert dt.read_status(ws) == 0
    assert np.all(np.abs(values(out) - o) <= _bound(o, mag, big, 64, L, "bf16"))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lens", [([3, 2], [1, 0]), ([200, 3], [150, 0]), ([1], [0])])
def test_rows_that_see_nothing_are_zero_and_others_stay(kind, rows, lens):
    """More rows than positions: the first rows sit before position 0."""
    g = np.random.default_rng(0)
    pool = Pool(g, lens, 16, 2, 64, "bf16")
    total = sum(rows) + 4
    start = (2 + np.concatenate([[0], np.cumsum(rows)])).astype(np.int32)
    q, q64 = _q(g, (total, 4, 64), kind)
    out = torch.full((total, 4, 64), 7.0, dtype=DTYPES[kind], device="cuda")
    ws = dt.workspace(dt.paged_attn_workspace_bytes(len(lens), total, 4, 2, 64))
    dt.paged_attn(q, cuda(start), pool.cache, cuda(pool.table), cuda(np.array(lens, np.int32)), 0.125,
                  out, ws, max_rows=max(rows))
    assert dt.read_status(ws) == 0
    got = values(out)
    assert np.all(got[:2] == 7) and np.all(got[-2:] == 7)
    for b, n in enumerate(rows):
        k, v = pool.rows(b, lens[b])
        o, mag, big = oracle.chunk(q64[start[b] : start[b + 1]], k, v, lens[b], 0, 0, 0.125)
        mine = got[start[b] : start[b + 1]]
        assert np.all(mine[: n - lens[b]] == 0)
        assert np.all(np.abs(mine - o) <= _bound(o, mag, big, 64, max(lens[b], 1), kind))


@pytest.mark.parametrize("n", [1, 30])
def test_strided_queries_and_a_loose_row_bound(n):
    _chunk(np.random.default_rng(n), [80, 300], [n, 1], 32, 8, 2, 64, "i8", "bf16", strided=True,
           max_rows=n + 500)


def test_large_scores_and_equal_scores():
    """The softmax keeps its maximum: scores of +-1000, and keys that are all alike."""
    g = np.random.default_rng(1)
    for n in (1, 70):
        pool = Pool(g, [400], 16, 2, 64, "bf16")
        pool.cache.k[:, 0] = pool.cache.k[0, 0, 0].clone()
        pool.host[0] = (values(pool.cache.k), None)
        q, q64 = _q(g, (n, 4, 64), "bf16")
        out = torch.zeros_like(q)
        ws = dt.workspace(dt.paged_attn_workspace_bytes(1, n, 4, 2, 64))
        dt.paged_attn(q, cuda(np.array([0, n], np.int32)), pool.cache, cuda(pool.table),
                      cuda(np.array([400], np.int32)), 40.0, out, ws, max_rows=n)
        k, v = pool.rows(0, 400)
        o, mag, big = oracle.chunk(q64, k, v, 400, 0, 0, 40.0)
        assert np.all(np.abs(values(out) - o) <= _bound(o, mag, big, 64, 400, "bf16"))


def test_long_context_is_split_and_joined():
    _chunk(np.random.default_rng(8), [40000, 7, 9000], [1, 1, 1], 64, 8, 1, 128, "e4m3", "bf16")
    _chunk(np.random.default_rng(9), [20011], [40], 64, 8, 2, 64, "bf16", "bf16")


# ---------------------------------------------------------------- trees --
def _tree(g, lens, nmax, page, hq, hkv, d, code, kind, window=0, sink=0, poison=False):
    pool = Pool(g, lens, page, hkv, d, code, poison)
    batch, rows = len(lens), nmax + 1
    n = g.integers(0, nmax + 1, batch).astype(np.int32)
    n[0] = nmax
    depth, anc = np.zeros((batch, nmax), np.int32), np.zeros((batch, nmax), np.uint64)
    for b in range(batch):
        _, depth[b, : n[b]], anc[b, : n[b]] = random_tree(g, n[b])
    q, q64 = _q(g, (batch, rows, hq, d), kind)
    kt, kt64 = _q(g, (batch, rows, hkv, d), kind)
    vt, vt64 = _q(g, (batch, rows, hkv, d), kind)
    if poison:  # rows behind a tree's last
        for b in range(batch):
            kt[b, n[b] + 1 :] = torch.nan
            vt[b, n[b] + 1 :] = torch.nan
    out = torch.full_like(q, 7.0)
    ws = dt.workspace(dt.verify_paged_workspace_bytes(batch, nmax, hq, hkv, d))
    scale = d ** -0.5
    dt.tree_verify_attn_paged(q, pool.cache, cuda(pool.table), cuda(np.array(lens, np.int32)), kt, vt,
                              cuda(anc.view(np.int64)), cuda(n), scale, out, ws,
                              depths=cuda(depth) if window else None, window=window, n_sink=sink)
    assert dt.read_status(ws) == 0
    got = values(out)
    for b, L in enumerate(lens):
        k, v = pool.rows(b, L)
        o, mag, big = oracle.tree(q64[b], k, v, kt64[b], vt64[b], anc[b], depth[b], n[b], L, window, sink,
                                  scale)
        tol = _bound(o, mag, big, d, L + rows, kind)
        err = np.abs(got[b, : n[b] + 1] - o)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        assert np.all(got[b, n[b] + 1 :] == 7)
    return pool, q, kt, vt, anc, n, got


@pytest.mark.parametrize("code", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("lens,nmax,page,hq,hkv,d", [
    ([0], 1, 16, 2, 2, 64), ([40, 300, 1], 8, 16, 8, 2, 64), ([100, 129], 32, 64, 32, 8, 128),
    ([500], 64, 128, 8, 2, 128), ([70, 0, 256, 17], 64, 8, 3, 1, 64), ([64], 3, 256, 8, 8, 128),
    ([90], 33, 32, 16, 1, 128)])
def test_tree_bf16(code, lens, nmax, page, hq, hkv, d):
    _tree(np.random.default_rng(nmax), lens, nmax, page, hq, hkv, d, code, "bf16")


@pytest.mark.parametrize("code", ["f32", "i8"])
@pytest.mark.parametrize("lens,nmax,page,hq,hkv,d", [([40, 300, 1], 8, 16, 8, 2, 64),
                                                    ([100, 129], 64, 64, 4, 4, 128)])
def test_tree_f32(code, lens, nmax, page, hq, hkv, d):
    _tree(np.random.default_rng(nmax), lens, nmax, page, hq, hkv, d, code, "f32")


@pytest.mark.parametrize("code", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sink", [(65, 0), (70, 4), (100, 300), (5000, 2)])
def test_tree_with_a_window(code, window, sink):
    _tree(np.random.default_rng(window), [300, 60, 700], 64, 32, 8, 2, 64, code, "bf16", window, sink)


@pytest.mark.parametrize("code", ["bf16", "e4m3", "i8"])
def test_tree_rows_and_slots_that_are_not_there_may_be_anything(code):
    _tree(np.random.default_rng(6), [50, 33, 200, 128], 20, 32, 8, 2, 128, code, "bf16", poison=True)


def test_paged_tree_equals_the_packed_one():
    """dt_tree_verify_attn on the rows that dt_kv_read unpacks, at bf16."""
    lens = [100, 333]
    pool, q, kt, vt, anc, n, got = _tree(np.random.default_rng(2), lens, 32, 16, 32, 8, 128, "bf16",
                                         "bf16")
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = (torch.zeros(sum(lens), 8, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    ws = dt.workspace(dt.verify_workspace_bytes(2, 32, 32, 8, 128, 333))
    dt.kv_read(pool.cache, cuda(pool.table), cuda(start), cuda(np.zeros(2, np.int32)), k, v, ws)
    out = torch.full_like(q, 7.0)
    dt.tree_verify_attn(q, k, v, cuda(start[:2].astype(np.int64)), cuda(np.array(lens, np.int32)), 333, kt,
                        vt, cuda(anc.view(np.int64)), cuda(n), 128 ** -0.5, out, ws)
    # two bf16 computations of the same sums, |v| up to 5: a few 2^-8 each
    assert np.abs(values(out) - got).max() < 0.05


# --------------------------------------------------- ways of being called --
@pytest.mark.parametrize("rows", [1, 50])
def test_graph_replay_with_new_lengths(rows):
    """One captured call serves other lengths, pages and queries."""
    g = np.random.default_rng(3)
    lens = [1500, 300]
    pool = Pool(g, lens, 32, 2, 64, "e4m3")
    q, _ = _q(g, (2 * rows, 8, 64), "bf16")
    out = torch.zeros_like(q)
    start, kv = cuda(np.array([0, rows, 2 * rows], np.int32)), cuda(np.array(lens, np.int32))
    table = cuda(pool.table)
    ws = dt.workspace(dt.paged_attn_workspace_bytes(2, 2 * rows, 8, 2, 64))
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        dt.paged_attn(q, start, pool.cache, table, kv, 0.125, out, ws, max_rows=rows)
    for now in (lens, [rows, 64], [700, 299]):
        qn, q64 = _q(g, (2 * rows, 8, 64), "bf16")
        q.copy_(qn)
        kv.copy_(cuda(np.array(now, np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            k, v = pool.rows(b, now[b])
            o, mag, big = oracle.chunk(q64[b * rows : (b + 1) * rows], k, v, now[b], 0, 0, 0.125)
            err = np.abs(values(out)[b * rows : (b + 1) * rows] - o)
            assert np.all(err <= _bound(o, mag, big, 64, now[b], "bf16"))
    assert dt.read_status(ws) == 0


@pytest.mark.parametrize("rows", [1, 60])
def test_the_same_call_gives_the_same_bits(rows):
    g = np.random.default_rng(4)
    lens = [5000, 20, 777]
    pool = Pool(g, lens, 64, 2, 128, "i8")
    n = [min(rows, x) for x in lens]
    start = cuda(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
    q, _ = _q(g, (sum(n), 8, 128), "bf16")
    ws = dt.workspace(dt.paged_attn_workspace_bytes(3, sum(n), 8, 2, 128))
    outs = []
    for _ in range(4):
        out = torch.zeros_like(q)
        dt.paged_attn(q, start, pool.cache, cuda(pool.table), cuda(np.array(lens, np.int32)), 0.1, out, ws,
                      max_rows=rows)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("rows", [1, 40])
def test_two_calls_at_once_on_two_streams(rows):
    g = np.random.default_rng(5)
    calls = []
    for seed in (1, 2):
        lens = [3000 * seed, 100]
        pool = Pool(g, lens, 64, 2, 64, "bf16")
        q, _ = _q(g, (2 * rows, 8, 64), "bf16")
        ws = dt.workspace(dt.paged_attn_workspace_bytes(2, 2 * rows, 8, 2, 64))
        calls.append((q, cuda(np.array([0, rows, 2 * rows], np.int32)), pool.cache, cuda(pool.table),
                      cuda(np.array(lens, np.int32)), ws, torch.cuda.Stream()))
    run = lambda c, out, s: dt.paged_attn(c[0], c[1], c[2], c[3], c[4], 0.125, out, c[5], max_rows=rows,
                                          stream=s)
    alone = []
    for c in calls:
        out = torch.zeros_like(c[0])
        run(c, out, None)
        alone.append(out)
    torch.cuda.synchronize()
    for _ in range(5):
        both = [torch.zeros_like(c[0]) for c in calls]
        torch.cuda.synchronize()
        for c, out in zip(calls, both):
            run(c, out, c[6])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, both))


@pytest.mark.parametrize("rows", [1, 20])
def test_impossible_lengths_are_recorded_and_leave_the_rows(rows):
    """Compared on the device before any use: nothing of such a request is read."""
    g = np.random.default_rng(6)
    pool = Pool(g, [64, 64], 16, 2, 64, "bf16")
    q, q64 = _q(g, (2 * rows, 4, 64), "bf16")
    ws = dt.workspace(dt.paged_attn_workspace_bytes(2, 2 * rows, 4, 2, 64))
    good = np.array([0, rows, 2 * rows], np.int32)
    for start, kv in ((good, [64, -1]), (good, [64, 65]), (np.array([0, rows, 2 * rows + 1], np.int32),
                                                          [64, 64])):
        out = torch.full_like(q, 7.0)
        dt.paged_attn(q, cuda(start), pool.cache, cuda(pool.table), cuda(np.array(kv, np.int32)), 0.125, out,
                      ws, max_rows=rows)
        assert dt.read_status(ws) == 6
        got = values(out)
        assert np.all(got[rows:] == 7)
        k, v = pool.rows(0, 64)
        o, mag, big = oracle.chunk(q64[:rows], k, v, 64, 0, 0, 0.125)
        assert np.all(np.abs(got[:rows] - o) <= _bound(o, mag, big, 64, 64, "bf16"))


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("code", ["bf16", "i8"])
def test_bad_pages_read_as_zeros(rows, code):
    g = np.random.default_rng(7)
    pool = Pool(g, [100], 16, 2, 64, code)
    q, q64 = _q(g, (rows, 4, 64), "bf16")
    ws = dt.workspace(dt.paged_attn_workspace_bytes(1, rows, 4, 2, 64))
    table = pool.table.copy()
    for bad in (-5, 10 ** 6):
        table[0, 2] = bad
        out = torch.zeros_like(q)
        dt.paged_attn(q, cuda(np.array([0, rows], np.int32)), pool.cache, cuda(table),
                      cuda(np.array([100], np.int32)), 0.125, out, ws, max_rows=rows)
        assert dt.read_status(ws) == 6
        k, v = pool.rows(0, 100)
        k[32:48] = 0
        v[32:48] = 0
        o, mag, big = oracle.chunk(q64, k, v, 100, 0, 0, 0.125)
        assert np.all(np.abs(values(out) - o) <= _bound(o, mag, big, 64, 100, "bf16"))


@pytest.mark.parametrize("code", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("d,batch,rows", [(128, 40, 16), (64, 50, 32), (128, 9, 200), (128, 60, 1)])
def test_many_tiles_on_every_sm_give_the_same_bits_and_are_right(code, d, batch, rows):
    """Every SM has several row tiles and hundreds of key tiles: what loads, converts, multiplies
    and sums runs at its own pace.  Repeats are equal, and a few requests are checked."""
    g = np.random.default_rng(batch)
    lens = [int(x) for x in g.integers(max(rows, 500), 3000, batch)]
    pool = Pool(g, lens, 64, 8, d, code)
    q, q64 = _q(g, (batch * rows, 32, d), "bf16")
    start, kv = cuda(np.arange(batch + 1, dtype=np.int32) * rows), cuda(np.array(lens, np.int32))
    table, ws = cuda(pool.table), dt.workspace(dt.paged_attn_workspace_bytes(batch, batch * rows, 32, 8, d))
    outs = []
    for _ in range(8):
        out = torch.zeros_like(q)
        dt.paged_attn(q, start, pool.cache, table, kv, d ** -0.5, out, ws, max_rows=rows)
        outs.append(out)
    assert dt.read_status(ws) == 0
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    got = values(outs[0])
    for b in g.integers(0, batch, 4):
        k, v = pool.rows(b, lens[b])
        pick = np.unique([0, rows // 2, rows - 1])
        ok = np.stack([oracle.seen_positions(lens[b] - rows + i, lens[b], 0, 0) for i in pick])
        o, mag, big = oracle.attend(q64[b * rows + pick], k, v, ok, d ** -0.5)
        err = np.abs(got[b * rows + pick] - o)
        assert np.all(err <= _bound(o, mag, big, d, lens[b], "bf16"))


# -------------------------------------------------- values nobody may see --
def _spoil(pool, b, j, page, value, code):
    """Position j of request b holds ``value`` in V (or, in a quantised cache, a scale of NaN)."""
    p, s = int(pool.table[b, j // page]), j % page
    if code == "bf16":
        pool.cache.v[p, :, s] = value
        pool.cache.k[p, :, s] = value
    else:
        pool.cache.v_scale[p, :, s] = float("nan")
        pool.cache.k_scale[p, :, s] = float("nan")


@pytest.mark.parametrize("code", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("n,lens", [(40, [300]), (5, [130]), (200, [1500]), (2, [9000])])
def test_a_position_that_is_not_a_number_reaches_only_the_rows_that_see_it(code, value, n, lens):
    """One late position of the chunk is spoilt: the rows before it share its tile with rows that
    see it, and their weight for it is 0.  They must be as if it were not there."""
    g = np.random.default_rng(n)
    page, L = 32, lens[0]
    pool = Pool(g, lens, page, 2, 64, code)
    k, v = pool.rows(0, L)
    first = L - n + n // 2                    # row n // 2 and later see the spoilt position
    _spoil(pool, 0, first, page, value, code)
    q, q64 = _q(g, (n, 8, 64), "bf16")
    out = torch.zeros_like(q)
    ws = dt.workspace(dt.paged_attn_workspace_bytes(1, n, 8, 2, 64))
    dt.paged_attn(q, cuda(np.array([0, n], np.int32)), pool.cache, cuda(pool.table),
                  cuda(np.array(lens, np.int32)), 0.125, out, ws, max_rows=n)
    assert dt.read_status(ws) == 0
    got = values(out)
    o, mag, big = oracle.chunk(q64, k, v, L, 0, 0, 0.125)
    clean = slice(0, n // 2)
    assert np.all(np.abs(got[clean] - o[clean]) <= _bound(o, mag, big, 64, L, "bf16")[clean])
    assert not np.any(np.isfinite(got[n // 2 :]).all(-1))


@pytest.mark.parametrize("code", ["bf16", "i8"])
def test_a_spoilt_position_behind_the_window(code):
    g = np.random.default_rng(3)
    L, n, page, window = 700, 70, 16, 100
    pool = Pool(g, [L], page, 2, 128, code)
    k, v = pool.rows(0, L)
    j = L - n - window + 30                   # rows 0 .. 29 see it, later ones do not
    _spoil(pool, 0, j, page, float("nan"), code)
    q, q64 = _q(g, (n, 4, 128), "bf16")
    out = torch.zeros_like(q)
    ws = dt.workspace(dt.paged_attn_workspace_bytes(1, n, 4, 2, 128))
    dt.paged_attn(q, cuda(np.array([0, n], np.int32)), pool.cache, cuda(pool.table),
                  cuda(np.array([L], np.int32)), 0.1, out, ws, max_rows=n, window=window)
    o, mag, big = oracle.chunk(q64, k, v, L, window, 0, 0.1)
    got, seen = values(out), np.array([oracle.seen_positions(L - n + i, L, window, 0)[j] for i in range(n)])
    assert seen[0] and not seen[-1]
    tol = _bound(o, mag, big, 128, L, "bf16")
    assert np.all(np.abs(got - o)[~seen] <= tol[~seen])
    assert not np.any(np.isfinite(got[seen]).all(-1))


@pytest.mark.parametrize("code", ["bf16", "e4m3"])
def test_a_tree_row_that_is_not_a_number_reaches_only_its_descendants(code):
    g = np.random.default_rng(4)
    L, nmax = 200, 12
    pool = Pool(g, [L], 32, 2, 64, code)
    _, depth, anc = random_tree(g, nmax)
    depth, anc = depth[None], anc[None]
    q, q64 = _q(g, (1, nmax + 1, 8, 64), "bf16")
    kt, kt64 = _q(g, (1, nmax + 1, 2, 64), "bf16")
    vt, vt64 = _q(g, (1, nmax + 1, 2, 64), "bf16")
    bad = 4                                   # node 4 = tree row 5
    vt[0, bad + 1] = float("nan")
    out = torch.zeros_like(q)
    ws = dt.workspace(dt.verify_paged_workspace_bytes(1, nmax, 8, 2, 64))
    dt.tree_verify_attn_paged(q, pool.cache, cuda(pool.table), cuda(np.array([L], np.int32)), kt, vt,
                              cuda(anc.view(np.int64)), cuda(np.array([nmax], np.int32)), 0.125, out, ws)
    k, v = pool.rows(0, L)
    o, mag, big = oracle.tree(q64[0], k, v, kt64[0], vt64[0], anc[0], depth[0], nmax, L, 0, 0, 0.125)
    got = values(out)[0]
    below = np.array([False] + [bool((int(a) >> bad) & 1) for a in anc[0]])
    tol = _bound(o, mag, big, 64, L + nmax + 1, "bf16")
    assert np.all(np.abs(got - o)[~below] <= tol[~below])
    assert below.sum() >= 1 and not np.any(np.isfinite(got[below]).all(-1))


# ------------------------------------------------------------ every code --
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("code", ["e4m3", "i8"])
def test_every_code_is_read_exactly(code, n):
    """Value column e of position j holds code (j + e) % 256; a query of zeros weighs all positions
    alike, so each output is a mean of known codes: only its own rounding, and that of the equal
    weights (times the one scale, a power of two: exact), is left."""
    L, page, d = 256, 64, 64
    codes = (np.arange(L)[:, None] + np.arange(d)[None]) % 256
    raw = codes.astype(np.uint8)
    if code == "e4m3":
        raw = np.where((raw & 0x7F) == 0x7F, raw & 0x80, raw)   # no NaN codes: dt_kv_write makes none
    t = torch.as_tensor(raw).view(DTYPES[code])
    val = t.float().double().numpy()
    cache = dt.KVCache.empty(L // page, page, 1, d, DTYPES[code])
    cache.v.view(torch.uint8).copy_(torch.as_tensor(raw).view(L // page, 1, page, d))
    cache.v_scale.fill_(0.25)
    cache.k_scale.fill_(1.0)
    q = torch.zeros(n, 2, d, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ws = dt.workspace(dt.paged_attn_workspace_bytes(1, n, 2, 1, d))
    table = cuda(np.arange(L // page, dtype=np.int32)[None])
    dt.paged_attn(q, cuda(np.array([0, n], np.int32)), cache, table, cuda(np.array([L], np.int32)), 0.1, out,
                  ws, max_rows=n)
    got = values(out)
    for i in range(n):
        seen = val[: L - n + i + 1] * 0.25
        o, mag = seen.mean(0), np.abs(seen).mean(0)
        assert np.all(np.abs(got[i] - o) <= 2.0 ** -8 * np.abs(o) + (L + 2) * 2.0 ** -24 * mag)


@pytest.mark.parametrize("rows", [1, 33])
@pytest.mark.parametrize("code", ["bf16", "i8"])
def test_a_cache_of_more_than_four_gigabytes(code, rows):
    """Pages at the far end of a large pool: offsets pass 32 bits."""
    g = np.random.default_rng(rows)
    page, hkv, d = 64, 2, 128
    pages = (5 << 30) // (page * hkv * d * (2 if code == "bf16" else 1))
    free = torch.cuda.mem_get_info()[0]
    assert free > 14 << 30
    small = Pool(g, [150], page, hkv, d, code)
    used = small.cache.k.shape[0]
    new = lambda t: None if t is None else torch.zeros(pages, *t.shape[1:], dtype=t.dtype, device="cuda")
    big = dt.KVCache(*(new(t) for t in (small.cache.k, small.cache.v, small.cache.k_scale,
                                        small.cache.v_scale)))
    for a, b in ((big.k, small.cache.k), (big.v, small.cache.v), (big.k_scale, small.cache.k_scale),
                 (big.v_scale, small.cache.v_scale)):
        if b is not None:
            a[pages - used :] = b
    q, q64 = _q(g, (rows, 8, d), "bf16")
    out = torch.zeros_like(q)
    ws = dt.workspace(dt.paged_attn_workspace_bytes(1, rows, 8, hkv, d))
    dt.paged_attn(q, cuda(np.array([0, rows], np.int32)), big, cuda(small.table + (pages - used)),
                  cuda(np.array([150], np.int32)), 0.1, out, ws, max_rows=rows)
    assert dt.read_status(ws) == 0
    k, v = small.rows(0, 150)
    o, mag, bigs = oracle.chunk(q64, k, v, 150, 0, 0, 0.1)
    assert np.all(np.abs(values(out) - o) <= _bound(o, mag, bigs, d, 150, "bf16"))


# ----------------------------------------------------- batches and shares --
@pytest.mark.parametrize("code,rows", [("bf16", 1), ("e4m3", 1), ("i8", 9), ("bf16", 40)])
def test_many_requests_of_very_different_lengths(code, rows):
    """More requests than a warp has lanes, some without rows, most of them short."""
    g = np.random.default_rng(11)
    lens = [int(x) for x in g.integers(1, 60, 150)] + [3000, 1, 700]
    n = [0 if i % 7 == 3 else min(x, rows) for i, x in enumerate(lens)]
    _chunk(g, lens, n, 16, 4, 2, 64, code, "bf16", max_rows=rows)


@pytest.mark.parametrize("hq,hkv", [(16, 1), (12, 1), (40, 2), (300, 1)])
@pytest.mark.parametrize("rows", [1, 2])
def test_group_sizes_at_the_kernels_borders(hq, hkv, rows):
    """8, 16 and 128 (row, head) pairs are where the kernels' tiles end."""
    _chunk(np.random.default_rng(hq), [200, 33], [rows, 1], 16, hq, hkv, 64, "i8", "bf16")


def test_a_window_over_shares_that_see_different_tiles():
    """First tokens, then a window far behind them, cut over many CTAs."""
    _chunk(np.random.default_rng(2), [20000], [3], 64, 32, 1, 128, "bf16", "bf16", 5000, 300)
    _chunk(np.random.default_rng(2), [9000], [150], 128, 4, 1, 64, "e4m3", "bf16", 3000, 200)


def test_another_device_s_workspace_and_cpu_tensors_are_refused():
    pool = Pool(np.random.default_rng(0), [20], 16, 2, 64, "bf16")
    q, _ = _q(np.random.default_rng(0), (1, 4, 64), "bf16")
    ws = dt.workspace(dt.paged_attn_workspace_bytes(1, 1, 4, 2, 64))
    start, table, kv = cuda(np.array([0, 1], np.int32)), cuda(pool.table), cuda(np.array([20], np.int32))
    call = lambda **kw: dt.paged_attn(*[{**dict(q=q, s=start, c=pool.cache, t=table, k=kv, x=0.1,
                                               o=torch.zeros_like(q), w=ws), **kw}[n] for n in "qsctkxow"],
                                      max_rows=1)
    call()
    for kw in (dict(w=ws.cpu()), dict(t=table.cpu()), dict(k=kv.cpu()), dict(q=q.cpu()), dict(o=q.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(dt.DtreeError):
        call(w=ws[:1024])
