"""fp64 attention over a paged key/value cache, and the cache's quantisation.

The cache keeps position p of request b in slot p % page_size of page
table[b][p // page_size]; pages are [n_pages, Hkv, page_size, d].  A row of
one head is stored as codes x * X / a with a = max(max |x|, 2^-100) and one
scale a / X (X = 448 for the 8-bit float, 127 for int8).

  chunk row i of n at position p = len - n + i sees the positions j <= p;
  with a window w > 0 only j > p - w or j < n_sink;
  tree row i (0 = the root, position len; node i - 1 at len + its depth) sees
  the cached positions under the same window, the root's tree row and the tree
  rows of its ancestors and itself.
A row that sees nothing is 0.
"""
import numpy as np

TINY = 2.0 ** -100


def quantise_row(x, top):
    """fp32 scale and the unrounded fp32 products x * (X / a) of one head row, as the fp32
    definition gives them; a row with an infinity or NaN has scale NaN and products 0."""
    x = np.asarray(x, np.float32)
    if not np.all(np.isfinite(x)):
        return np.float32(np.nan), np.zeros_like(x)
    a = np.maximum(np.abs(x).max(), np.float32(TINY))
    return a / np.float32(top), x * (np.float32(top) / a)


def seen_positions(p, length, window, n_sink):
    """Cached positions that a row at position p sees, as a boolean [length]."""
    j = np.arange(length)
    ok = j <= p
    if window:
        ok &= (j > p - window) | (j < n_sink)
    return ok


def gather(pages, scale, table, length):
    """fp64 rows [length, Hkv, d] of a request's positions."""
    ps = pages.shape[2]
    j = np.arange(length)
    x = pages[table[j // ps], :, j % ps].astype(np.float64)
    if scale is not None:
        x = x * scale[table[j // ps], :, j % ps].astype(np.float64)[..., None]
    return x


def attend(q, k, v, ok, scale):
    """q [R, Hq, d], k/v [L, Hkv, d], ok [R, L]: outputs [R, Hq, d], the weighted sums of |v|, and
    the largest sum of |q k| over a row's visible keys (for error bounds)."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    R, Hq, d = q.shape
    G = Hq // k.shape[1]
    out, mag, big = np.zeros((R, Hq, d)), np.zeros((R, Hq, d)), np.zeros((R, Hq))
    for i in range(R):
        js = np.nonzero(ok[i])[0]
        if len(js) == 0:
            continue
        for h in range(Hq):
            kk, vv = k[js, h // G], v[js, h // G]
            s = scale * (kk @ q[i, h])
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ vv
            mag[i, h] = w @ np.abs(vv)
            big[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, mag, big


def chunk(q, k, v, length, window, n_sink, scale):
    """One request's chunk: its rows are the last positions of ``length``."""
    n = q.shape[0]
    ok = np.stack([seen_positions(length - n + i, length, window, n_sink) for i in range(n)])
    return attend(q, k, v, ok, scale)


def tree(q, k, v, k_tree, v_tree, anc, depths, n, length, window, n_sink, scale):
    """One request's n + 1 tree rows over ``length`` cached positions."""
    rows = []
    for i in range(n + 1):
        p = length + (0 if i == 0 else int(depths[i - 1]))
        own = np.zeros(n + 1, bool)
        own[0] = True
        if i:
            for j in range(n):
                own[j + 1] = (int(anc[i - 1]) >> j) & 1
        rows.append(np.concatenate([seen_positions(p, length, window, n_sink), own]))
    return attend(q[: n + 1], np.concatenate([k, k_tree[: n + 1]]),
                  np.concatenate([v, v_tree[: n + 1]]), np.stack(rows), scale)
