"""GPU tests of dt_logits_process against fp64.

Error bound: at most five fp32 roundings on a value whose largest magnitude on
the way is M, and one more at the end: 6 * 2^-24 M, plus 2^-8 |z| for bf16.
Untouched values are copied bit by bit.
"""
import numpy as np
import pytest
import torch

from oracle import logits as oracle
from tests.serving_util import DTYPES, cuda, random_tree, values

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import draft_tree_construction_markov_b200 as dt


def _i32(a):
    return cuda(np.asarray(a, np.int32))


class Case:
    def __init__(self, seed, batch, nmax, V, kind, hist, bias=3, mask=True, penal=True):
        g = self.g = np.random.default_rng(seed)
        self.batch, self.nmax, self.V, self.kind = batch, nmax, V, kind
        rows = nmax + 1
        self.logits = torch.as_tensor((3 * g.standard_normal((batch, rows, V))).astype(np.float32)
                                      ).to(DTYPES[kind])
        self.n = g.integers(0, nmax + 1, batch)
        self.n[0] = nmax
        tok = lambda k: np.where(g.random(k) < 0.5, g.integers(0, min(V, 5), k), g.integers(0, V, k))
        self.anc, self.parent = np.zeros((batch, max(nmax, 1)), np.uint64), []
        for b in range(batch):
            p, _, a = random_tree(g, self.n[b])
            self.parent.append(p)
            self.anc[b, : self.n[b]] = a
        self.tokens = tok((batch, max(nmax, 1)))
        self.hist = [tok(n) for n in hist]
        self.n_prompt = np.array([g.integers(0, n + 1) for n in hist])
        self.penal = penal
        self.rho, self.pres, self.freq = g.uniform(0.7, 1.5, batch), g.uniform(-1, 1, batch), \
            g.uniform(-0.5, 0.5, batch)
        self.bias = [[(int(g.integers(0, V)), float(g.standard_normal() * 5)) for _ in range(bias)]
                     for _ in range(batch)]
        if bias:
            self.bias[0][-1] = (self.bias[0][0][0], 2.5)   # listed twice: the last counts
        self.mask = self.mask_row = None
        if mask:
            self.mask = g.random((batch * rows + 1, V)) < g.choice([0.03, 0.97], (batch * rows + 1, 1))
            self.mask[0] = False                           # everything forbidden
            self.mask_row = g.integers(-1, batch * rows + 1, (batch, rows))

    def words(self):
        pad = np.zeros((self.mask.shape[0], -(-self.V // 32) * 32), bool)
        pad[:, : self.V] = self.mask
        return cuda(np.packbits(pad, axis=1, bitorder="little").view(np.int32))

    def args(self):
        start = lambda x: _i32(np.concatenate([[0], np.cumsum([len(y) for y in x])]))
        f = lambda x: cuda(np.asarray(x, np.float32))
        a = {}
        if self.nmax:
            a.update(tokens=_i32(self.tokens), anc=cuda(self.anc.view(np.int64)), n_nodes=_i32(self.n))
        a.update(history=_i32(np.concatenate(self.hist)), history_start=start(self.hist),
                 n_prompt=_i32(self.n_prompt))
        if self.penal:
            a.update(repetition=f(self.rho), presence=f(self.pres), frequency=f(self.freq))
        flat = [e for b in self.bias for e in b]
        if flat:
            a.update(bias_start=start(self.bias), bias_token=_i32([e[0] for e in flat]),
                     bias_value=f([e[1] for e in flat]))
        if self.mask is not None:
            a.update(mask=self.words(), mask_row=_i32(self.mask_row))
        return a

    def check(self, out, before):
        got, src = values(out), values(self.logits)
        f32 = lambda x: float(np.float32(x))
        for b in range(self.batch):
            for i in range(self.nmax + 1):
                if i > self.n[b]:
                    assert torch.equal(out[b, i].cpu(), before[b, i])
                    continue
                path, j = [], i - 1
                while j >= 0:
                    path.append(self.tokens[b, j])
                    j = self.parent[b][j]
                m = None if self.mask is None else self.mask_row[b, i]
                allowed = None if m is None or m < 0 else self.mask[m]
                np_ = self.n_prompt[b]
                par = (f32(self.rho[b]), f32(self.pres[b]), f32(self.freq[b])) if self.penal else (1, 0, 0)
                z, big = oracle.process_row(src[b, i], self.hist[b][:np_], self.hist[b][np_:], path, *par,
                                            [(t, f32(y)) for t, y in self.bias[b]], allowed)
                fin = np.isfinite(z)
                assert np.array_equal(got[b, i] == -np.inf, ~fin)
                tol = 6 * 2.0 ** -24 * big
                if self.kind == "bf16":
                    tol = tol + 2.0 ** -8 * (np.abs(z) + tol)
                assert np.all(np.abs(got[b, i] - z)[fin] <= tol[fin])
                same = fin & (z == src[b, i])
                assert np.array_equal(got[b, i][same], src[b, i][same])


def _run(c, in_place, **more):
    x = c.logits.cuda()
    out = x if in_place else torch.full_like(x, 7.0)
    before = out.cpu().clone()
    ws = dt.workspace(dt.logits_workspace_bytes())
    dt.logits_process(x, out, ws, **{**c.args(), **more})
    assert dt.read_status(ws) == 0
    return out, before


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("batch,nmax,V,hist", [
    (1, 0, 1, [4]), (2, 0, 7, [0, 3]), (3, 8, 512, [20, 0, 300]), (2, 64, 1003, [5, 1000]),
    (1, 3, 4089, [50]), (1, 5, 4096, [2000]), (2, 4, 8195, [700, 9]), (5, 1, 32003, [1, 2, 3, 4, 5]),
    (1, 2, 12288, [10000])])
def test_logits_match_the_definition(in_place, kind, batch, nmax, V, hist):
    c = Case(V + nmax, batch, nmax, V, kind, hist)
    c.check(*_run(c, in_place))


@pytest.mark.parametrize("in_place", [False, True])
def test_at_the_round_s_vocabulary(in_place):
    c = Case(3, 2, 4, 151936, "bf16", [3000, 100], bias=50)
    c.check(*_run(c, in_place))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_each_part_alone(kind):
    c = Case(1, 2, 6, 777, kind, [40, 9], bias=0, mask=False)
    c.check(*_run(c, False))
    c = Case(2, 2, 6, 777, kind, [40, 9], bias=5, mask=False, penal=False)
    c.check(*_run(c, False))
    c = Case(3, 2, 6, 777, kind, [0, 0], bias=0, mask=True, penal=False)
    c.check(*_run(c, True))


def test_masks_by_row_when_no_index_is_given():
    c = Case(4, 2, 3, 100, "f32", [5, 5])
    c.mask = c.mask[:8]
    a = c.args()
    a.pop("mask_row")
    c.mask_row = np.arange(8).reshape(2, 4)
    x = c.logits.cuda()
    out = torch.full_like(x, 7.0)
    ws = dt.workspace(dt.logits_workspace_bytes())
    dt.logits_process(x, out, ws, **a)
    c.check(out, torch.full_like(c.logits, 7.0))


def test_infinities_and_nan_pass_through():
    V = 64
    x = torch.zeros(1, 1, V)
    x[0, 0, :4] = torch.tensor([np.inf, -np.inf, np.nan, -np.inf])
    d, out = x.cuda(), torch.zeros(1, 1, V, device="cuda")
    ws = dt.workspace(dt.logits_workspace_bytes())
    mask = torch.full((1, 2), -1, dtype=torch.int32)
    mask[0, 0] = ~(1 << 2)                                # token 2 (a NaN) is forbidden
    dt.logits_process(d, out, ws, history=_i32([0, 1, 3]), history_start=_i32([0, 3]),
                      repetition=cuda(np.array([1.5], np.float32)),
                      frequency=cuda(np.array([0.5], np.float32)), mask=mask.cuda())
    assert out[0, 0, :4].tolist() == [np.inf, -np.inf, -np.inf, -np.inf]
    assert torch.all(out[0, 0, 4:] == 0)


def test_what_is_out_of_range_is_ignored_and_recorded():
    """Compared on the device before any use."""
    V = 50
    x = torch.arange(2 * V, dtype=torch.float32).reshape(1, 2, V).cuda()
    tree = dict(tokens=_i32([[99]]), anc=cuda(np.ones((1, 1), np.int64)), n_nodes=_i32([1]))
    one = lambda v: cuda(np.array([v], np.float32))
    ws = dt.workspace(dt.logits_workspace_bytes())
    bad = [dict(tree), dict(history=_i32([-1, 60]), history_start=_i32([0, 2]), frequency=one(1.0)),
           dict(history=_i32([1, 2]), history_start=_i32([0, 3]), frequency=one(1.0)),
           dict(history=_i32([1, 2]), history_start=_i32([1, 0]), frequency=one(1.0)),
           dict(bias_token=_i32([50]), bias_value=one(2.0), bias_start=_i32([0, 1])),
           dict(mask=_i32([[0, 0]]), mask_row=_i32([[1, -2]]))]
    for b in bad:
        out = torch.zeros_like(x)
        if "tokens" not in b:
            b.update(tree, tokens=_i32([[3]]))
        dt.logits_process(x, out, ws, **b)
        assert dt.read_status(ws) == 6
        want = x.clone()
        if "frequency" in b:
            want[0, 1, 3] -= 1               # the row's own path token still counts
        assert torch.equal(out, want)
    out = torch.zeros_like(x)
    dt.logits_process(x, out, ws, **{**tree, "tokens": _i32([[3]]), "n_nodes": _i32([5])})
    assert dt.read_status(ws) == 6 and torch.equal(out, x)


def test_no_lists_copies_and_a_graph_replays():
    x = torch.randn(2, 1, 1001, dtype=torch.float32, device="cuda").to(torch.bfloat16)
    out = torch.zeros_like(x)
    ws = dt.workspace(dt.logits_workspace_bytes())
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    dt.logits_process(x, out, ws, history=empty, history_start=_i32([0, 0, 0]))
    assert torch.equal(out, x)
    h = _i32([5, 6, 7])
    a = dict(history=h, history_start=_i32([0, 2, 3]), frequency=cuda(np.ones(2, np.float32)))
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        dt.logits_process(x, out, ws, **a)
    for hist in ([5, 6, 7], [1000, 1000, 0]):
        h.copy_(_i32(hist))
        graph.replay()
        torch.cuda.synchronize()
        want = x.float().cpu()
        for b, t in ((0, hist[:2]), (1, hist[2:])):
            for v in t:
                want[b, 0, v] -= 1
        assert torch.equal(out.cpu(), want.to(torch.bfloat16))
