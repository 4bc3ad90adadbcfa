"""GPU tests of when the paged attention does rows again key by key, and of what that gives.

A row is done again where a value that it does not see may have made its sums infinite or NaN.  That
form takes a hundred times as long as the tiles, so the calls below are timed beside the same call on
a pool without the odd value: three times as long, and half a millisecond, is let pass (the timer and
the look at the outputs); rows done again for nothing would take many milliseconds.
"""
import numpy as np
import pytest
import torch

from oracle import paged_attn as oracle
from tests.serving_util import cuda, random_tree, values
from tests.test_gpu_paged_attn import Pool, _bound, _q

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import draft_tree_construction_markov_b200 as dt


def _ms(call):
    """The fastest of several calls."""
    best = float("inf")
    for _ in range(6):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


class Chunk:
    def __init__(self, g, lens, rows, code, hq=8, hkv=2, d=128, page=64, window=0, sink=0):
        self.lens, self.rows, self.code, self.page, self.d = lens, rows, code, page, d
        self.window, self.sink = window, sink
        self.pool = Pool(g, lens, page, hkv, d, code)
        n = len(lens)
        self.q, self.q64 = _q(g, (n * rows, hq, d), "bf16")
        self.out = torch.zeros_like(self.q)
        self.ws = dt.workspace(dt.paged_attn_workspace_bytes(n, n * rows, hq, hkv, d))
        self.args = (cuda(np.arange(n + 1, dtype=np.int32) * rows), self.pool.cache, cuda(self.pool.table),
                     cuda(np.array(lens, np.int32)))

    def __call__(self):
        dt.paged_attn(self.q, *self.args, self.d ** -0.5, self.out, self.ws, max_rows=self.rows,
                      window=self.window, n_sink=self.sink)

    def ms(self):
        self()
        assert dt.read_status(self.ws) == 0
        return _ms(self)

    def check(self, b, k, v, pick, ok=None):
        """Rows pick of request b against fp64."""
        L = self.lens[b]
        see = np.stack([oracle.seen_positions(L - self.rows + i, L, self.window, self.sink) for i in pick])
        o, mag, big = oracle.attend(self.q64[b * self.rows + pick], k, v, see, self.d ** -0.5)
        err = np.abs(values(self.out)[b * self.rows + pick] - o)
        assert np.all(err <= _bound(o, mag, big, self.d, L, "bf16"))


def _unused(pool, lens, page):
    """[page, slot] of the pool's places that hold no request's position."""
    free = torch.ones(pool.cache.k.shape[0], page, dtype=torch.bool)
    for b, L in enumerate(lens):
        for p in range(L):
            free[pool.table[b, p // page], p % page] = False
    return free.cuda()


def _nan_scales(pool, lens, page):
    hole = _unused(pool, lens, page)[:, None].expand(pool.cache.k.shape[:3])
    for s in (pool.cache.k_scale, pool.cache.v_scale):
        s[hole] = float("nan")


@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("rows", [1, 6, 30, 200])
def test_scales_of_slots_without_a_position_cost_nothing(code, rows):
    """As a pool that was never cleared has them, or a page whose former owner was not finite."""
    lens = [3000, 2111, 1500]
    c = Chunk(np.random.default_rng(rows), lens, rows, code)
    clean = c.ms()
    _nan_scales(c.pool, lens, c.page)
    assert c.ms() <= 3 * clean + 0.5
    for b in (0, 1, 2):
        c.check(b, *c.pool.rows(b, lens[b]), np.unique([0, rows // 2, rows - 1]))


@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("nmax", [20, 64])
def test_such_scales_beside_a_tree(code, nmax):
    g = np.random.default_rng(nmax)
    lens, page, hq, hkv, d = [2501, 1033], 64, 8, 2, 128
    pool = Pool(g, lens, page, hkv, d, code)
    n = np.array([nmax, nmax // 2], np.int32)
    depth, anc = np.zeros((2, nmax), np.int32), np.zeros((2, nmax), np.uint64)
    for b in range(2):
        _, depth[b, : n[b]], anc[b, : n[b]] = random_tree(g, n[b])
    q, q64 = _q(g, (2, nmax + 1, hq, d), "bf16")
    kt, kt64 = _q(g, (2, nmax + 1, hkv, d), "bf16")
    vt, vt64 = _q(g, (2, nmax + 1, hkv, d), "bf16")
    out = torch.zeros_like(q)
    ws = dt.workspace(dt.verify_paged_workspace_bytes(2, nmax, hq, hkv, d))
    args = (cuda(pool.table), cuda(np.array(lens, np.int32)), kt, vt, cuda(anc.view(np.int64)), cuda(n))
    call = lambda: dt.tree_verify_attn_paged(q, pool.cache, *args, d ** -0.5, out, ws)
    call()
    clean = _ms(call)
    _nan_scales(pool, lens, page)
    call()
    assert _ms(call) <= 3 * clean + 0.5
    assert dt.read_status(ws) == 0
    for b, L in enumerate(lens):
        o, mag, big = oracle.tree(q64[b], *pool.rows(b, L), kt64[b], vt64[b], anc[b], depth[b], n[b], L, 0, 0,
                                  d ** -0.5)
        err = np.abs(values(out)[b, : n[b] + 1] - o)
        assert np.all(err <= _bound(o, mag, big, d, L + nmax + 1, "bf16"))


@pytest.mark.parametrize("code", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("rows,at", [(1, 900), (4, 900), (4, 7990), (40, 100), (200, 2900)])
def test_what_every_row_sees_is_not_done_again(code, rows, at):
    """A position that is not a number and that all rows of the request see: NaN it is, at once.
    (A bf16 cache: in one column, and the others are as they would be without it.)"""
    lens = [8000, 3000] if rows < 40 else [4000, 3000]
    c = Chunk(np.random.default_rng(at), lens, rows, code)
    k, v = c.pool.rows(0, lens[0])
    clean = c.ms()
    p, s = int(c.pool.table[0, at // c.page]), at % c.page
    if code == "bf16":
        c.pool.cache.v[p, :, s, 5] = float("nan")
    else:
        c.pool.cache.v_scale[p, :, s] = float("nan")
    assert c.ms() <= 3 * clean + 0.5
    got = values(c.out)
    nan = np.isnan(got[:rows])
    assert np.isfinite(got[rows:]).all()
    if code != "bf16":
        assert nan.all()
        return
    assert nan[..., 5].all() and not np.delete(nan, 5, -1).any()
    pick = np.unique([0, rows // 2, rows - 1])
    see = np.stack([oracle.seen_positions(lens[0] - rows + i, lens[0], 0, 0) for i in pick])
    o, mag, big = oracle.attend(c.q64[pick], k, v, see, c.d ** -0.5)
    err = np.delete(np.abs(got[pick] - o) - _bound(o, mag, big, c.d, lens[0], "bf16"), 5, -1)
    assert np.all(err <= 0)


@pytest.mark.parametrize("window,sink,at", [(1000, 0, 4000 - 4 - 1000), (1000, 70, 69), (1000, 70, 70),
                                            (333, 5, 4000 - 2 - 333)])
@pytest.mark.parametrize("rows,hq,hkv", [(4, 8, 2), (1, 8, 2), (60, 8, 1)])
def test_a_hidden_position_at_the_ends_of_what_a_tile_reads(window, sink, at, rows, hq, hkv):
    """Just before the window, or at the end of the first tokens: in the tile, seen by some rows or
    by none.  Rows that do not see it are as if it were not there; the others are NaN."""
    c = Chunk(np.random.default_rng(at), [4000], rows, "bf16", hq, hkv, window=window, sink=sink)
    k, v = c.pool.rows(0, 4000)
    p, s = int(c.pool.table[0, at // c.page]), at % c.page
    c.pool.cache.v[p, :, s] = float("nan")
    c()
    assert dt.read_status(c.ws) == 0
    got = values(c.out)
    see = np.stack([oracle.seen_positions(4000 - rows + i, 4000, window, sink) for i in range(rows)])
    o, mag, big = oracle.attend(c.q64, k, v, see, c.d ** -0.5)
    hit = see[:, at]
    assert np.isnan(got[hit]).all()
    assert np.all(np.abs(got - o)[~hit] <= _bound(o, mag, big, c.d, 4000, "bf16")[~hit])


@pytest.mark.parametrize("rows", [2, 5])
def test_whole_tiles_of_many_requests_with_a_hidden_position(rows):
    """So many requests that a worker has whole row tiles, in each a position that only the first
    rows see."""
    lens = [200] * 900
    c = Chunk(np.random.default_rng(rows), lens, rows, "bf16", d=64, window=100)
    k, v = c.pool.rows(7, 200)
    at = 200 - rows - 100 + 1               # row 0 sees it, at the start of its window
    for b in range(900):
        c.pool.cache.v[int(c.pool.table[b, at // c.page]), :, at % c.page] = float("nan")
    c()
    assert dt.read_status(c.ws) == 0
    got = torch.isnan(c.out).view(900, rows, -1)
    assert got[:, 0].all() and not got[:, 1:].any()
    c.check(7, k, v, np.arange(1, rows))


@pytest.mark.parametrize("rows", [2, 5])
def test_sums_that_pass_fp32_only_over_the_maximum_in_use(rows):
    """Weights may be 2^8 over the maximum in use.  Where a sum passes fp32 for that alone, the row is
    done again: values of 2^119, and late keys that score 5 (7.2 in log2) over the others: 150 + 48 * 148
    weights pass 2^128; relative to the largest score so far they are never more than 160, and
    160 * 2^119 < 2^127.  All values are alike, so the output is that value, but for the roundings of
    the weights and of the output (2^-8 each) and fp32 sums."""
    c = Chunk(np.random.default_rng(rows), [200] * 900, rows, "bf16", d=64)
    c.pool.cache.v.fill_(2.0 ** 119)
    c.pool.cache.k.zero_()
    for b in range(900):
        for p in range(2, 4):               # positions 150 to 199 on pages of 64
            c.pool.cache.k[int(c.pool.table[b, p]), :, max(150 - 64 * p, 0) :, 0] = 5.0
    c.q.zero_()
    c.q[..., 0] = 8.0
    c()
    assert dt.read_status(c.ws) == 0
    got = values(c.out)
    assert np.all(np.abs(got - 2.0 ** 119) <= 2.0 ** 119 * (2.0 ** -7 + 2.0 ** -14))


@pytest.mark.parametrize("seed", [1, 2])
def test_a_code_that_is_no_number_counts_alike_in_a_row_done_again(seed):
    """The e4m3 codes 0x7f and 0xff count as +-480, in K and in V: also for a tree row that is done
    again because of a row of the tree that it does not see."""
    g = np.random.default_rng(seed)
    L, nmax, hq, hkv, d, page = 100, 12, 4, 1, 64, 32
    pool = Pool(g, [L], page, hkv, d, "e4m3")
    for t, cols in ((pool.cache.k, 3), (pool.cache.v, 7)):
        t.view(torch.uint8)[:, :, 5, cols] = 0x7F
        t.view(torch.uint8)[:, :, 9, cols] = 0xFF
    # small keys' scales: a score of 480 must not take the whole softmax
    pool.cache.k_scale.mul_(0.02)
    host = []
    for t, s in ((pool.cache.k, pool.cache.k_scale), (pool.cache.v, pool.cache.v_scale)):
        x = t.float().cpu()
        x[:, :, 5] = torch.nan_to_num(x[:, :, 5], nan=480.0)
        x[:, :, 9] = torch.nan_to_num(x[:, :, 9], nan=-480.0)
        host.append((x.double().numpy(), values(s)))
    k, v = (oracle.gather(x, s, pool.table[0], L) for x, s in host)
    _, depth, anc = random_tree(g, nmax)
    q, q64 = _q(g, (1, nmax + 1, hq, d), "bf16")
    kt, kt64 = _q(g, (1, nmax + 1, hkv, d), "bf16")
    vt, vt64 = _q(g, (1, nmax + 1, hkv, d), "bf16")
    bad = 4
    vt[0, bad + 1] = float("nan")
    out = torch.zeros_like(q)
    ws = dt.workspace(dt.verify_paged_workspace_bytes(1, nmax, hq, hkv, d))
    dt.tree_verify_attn_paged(q, pool.cache, cuda(pool.table), cuda(np.array([L], np.int32)), kt, vt,
                              cuda(anc[None].view(np.int64)), cuda(np.array([nmax], np.int32)), 0.125, out, ws)
    o, mag, big = oracle.tree(q64[0], k, v, kt64[0], vt64[0], anc, depth, nmax, L, 0, 0, 0.125)
    below = np.array([False] + [bool((int(a) >> bad) & 1) for a in anc])
    tol = _bound(o, mag, big, d, L + nmax + 1, "bf16")
    assert (~below).sum() >= 2
    assert np.all(np.abs(values(out)[0] - o)[~below] <= tol[~below])


@pytest.mark.parametrize("late", [False, True])
def test_long_rows_done_again_hold_no_worker_up(late):
    """420 requests of 16 (row, head) pairs share one context of 250 thousand positions, so that a
    worker has whole row tiles.  A position that is not a number, seen by all rows or (the last one)
    by half of them: no wait may run out meanwhile, and rows that do not see it are as they were."""
    g = np.random.default_rng(1)
    L, batch, rows, hkv, d, page = 250000 if not late else 60000, 420, 2, 8, 64, 256
    pages = -(-L // page)
    cache = dt.KVCache.empty(pages, page, hkv, d, torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    cache.k.normal_(generator=gen)
    cache.v.normal_(generator=gen)
    flat = lambda t: values(t.transpose(1, 2).reshape(-1, hkv, d)[:L])
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
    q, q64 = _q(g, (batch * rows, 64, d), "bf16")
    out = torch.zeros_like(q)
    at = L - 1 if late else 5
    k, v = flat(cache.k), flat(cache.v)
    cache.v[at // page, :, at % page, 3] = float("nan")
    ws = dt.workspace(dt.paged_attn_workspace_bytes(batch, batch * rows, 64, hkv, d))
    dt.paged_attn(q, cuda(np.arange(batch + 1, dtype=np.int32) * rows), cache, table,
                  cuda(np.full(batch, L, np.int32)), 0.125, out, ws, max_rows=rows)
    assert dt.read_status(ws) == 0
    got = torch.isnan(out).view(batch, rows, 64, d)
    assert got[:, 1, :, 3].all() and got[:, 0, :, 3].all() != late
    got[..., 3] = False
    assert not got.any()
    b = 200
    see = np.stack([oracle.seen_positions(L - rows + i, L, 0, 0) for i in range(rows)])
    o, mag, big = oracle.attend(q64[b * rows : (b + 1) * rows, :8], k[:, :1], v[:, :1], see, 0.125)
    err = np.abs(values(out)[b * rows : (b + 1) * rows, :8] - o) - _bound(o, mag, big, d, L, "bf16")
    assert np.all(np.delete(err, 3, -1) <= 0)
    if late:
        assert np.all(err[0] <= 0)


@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("rows,L", [(1, 33), (1, 500), (4, 500), (20, 500)])
def test_a_seen_score_of_minus_infinity_takes_its_value_s_scale(code, rows, L):
    """A key's scale is infinite and its value's is not a number: whatever the sign of the score (a
    weight of 0 for some heads), the rows that see the position are NaN, and the others are not."""
    c = Chunk(np.random.default_rng(L + rows), [L], rows, code)
    k, v = c.pool.rows(0, L)
    at = L - 1 if rows == 1 else L - 2
    p, s = int(c.pool.table[0, at // c.page]), at % c.page
    c.pool.cache.k_scale[p, :, s] = float("inf")
    c.pool.cache.v_scale[p, :, s] = float("nan")
    c()
    assert dt.read_status(c.ws) == 0
    nan = torch.isnan(c.out).flatten(1)
    hit = torch.arange(rows, device="cuda") >= rows - (L - at)
    assert nan[hit].all() and not nan[~hit].any()
    if rows > 2:
        c.check(0, k, v, np.arange(rows - 2))
