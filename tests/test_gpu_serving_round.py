"""The serving operators together, as a decode loop uses them.

A one-layer target (embedding -> q, k, v; grouped attention; output projection)
takes a prompt in two chunks (kv_write, paged_attn), then runs rounds: tree_build
drafts, tree_verify_attn_paged verifies over the paged cache, logits_process
applies the request's penalties along every path, tree_accept walks greedily,
kv_commit keeps what was accepted.  Greedy acceptance is lossless, so every
emitted token has to be the argmax that step-by-step decoding would take: the
reference recomputes each step in fp64 from the emitted tokens alone.
"""
import numpy as np
import pytest
import torch

from gen import make_workload
from oracle import logits as olog
from oracle import paged_attn as oattn
from tests.serving_util import DTYPES, cuda, page_table, to_codes, values

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import draft_tree_construction_markov_b200 as dt
    from tests.gpu_util import build_inputs

HQ, HKV, D = 4, 2, 64


def _target(V, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    E = r(V, 64)
    bf = lambda x: x.to(torch.bfloat16)
    return dict(q=bf(E @ r(64, HQ * D) / 8).view(V, HQ, D), k=bf(E @ r(64, HKV * D) / 8).view(V, HKV, D),
                v=bf(E @ r(64, HKV * D) / 8).view(V, HKV, D), w=bf(r(HQ * D, V) / 2))


@pytest.mark.parametrize("code", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("window,sink", [(0, 0), (24, 4)])
def test_rounds_emit_what_step_by_step_decoding_would(code, window, sink):
    w = make_workload("tiny", seed=3, batch=3, N=8)
    V, batch, Nmax, Bk = w.V, w.batch, w.Nmax, w.Bk
    g = np.random.default_rng(1)
    m = _target(V, 5)
    dm = {k: t.cuda() for k, t in m.items()}
    scale, page, rounds = D ** -0.5, 8, 4
    prompts = [g.integers(0, V, n).tolist() for n in (40, 7, 23)]
    cap = [len(p) + rounds * (Bk + 1) + 1 for p in prompts]
    table, pool = page_table(g, cap, page)
    cache, dtable = dt.KVCache.empty(pool, page, HKV, D, DTYPES[code]), cuda(table)
    i32 = lambda a: cuda(np.asarray(a, np.int32))
    ws = dt.workspace(max(dt.kv_workspace_bytes(), dt.paged_attn_workspace_bytes(batch, 128, HQ, HKV, D),
                          dt.verify_paged_workspace_bytes(batch, Nmax, HQ, HKV, D),
                          dt.accept_workspace_bytes(batch, Nmax, V),
                          dt.build_workspace_bytes(batch, Bk, V, w.r, w.k, Nmax)))

    # the prompt in two chunks; all its tokens but the last (the first round's root) enter the cache
    have = [0] * batch
    for part in (0, 1):
        ends = [(len(p) - 1) // 2 if part == 0 else len(p) - 1 for p in prompts]
        toks = [t for b, p in enumerate(prompts) for t in p[have[b] : ends[b]]]
        start = i32(np.concatenate([[0], np.cumsum([ends[b] - have[b] for b in range(batch)])]))
        ix = torch.tensor(toks).cuda()
        dt.kv_write(dm["k"][ix], dm["v"][ix], start, i32(have), cache, dtable, ws)
        out = torch.zeros(len(toks), HQ, D, dtype=torch.bfloat16, device="cuda")
        dt.paged_attn(dm["q"][ix], start, cache, dtable, i32(ends), scale, out, ws, max_rows=64,
                      window=window, n_sink=sink)
        at = 0
        for b, p in enumerate(prompts):
            n = ends[b] - have[b]
            o, mag = _reference(m, p[: ends[b]], n, code, window, sink, scale)
            err = np.abs(values(out)[at : at + n] - o)
            assert np.all(err <= 2.0 ** -7 * (np.abs(o) + mag) * 1.01)
            at += n
        have = ends

    rho, pres, freq = (cuda(g.uniform(*r, batch).astype(np.float32)) for r in
                       ((1.0, 1.4), (0.0, 0.5), (0.0, 0.5)))
    emitted = [list() for _ in prompts]
    x = build_inputs(w)
    tree = dt.Tree.empty(batch, Nmax, V)
    acc, n_acc, bonus = i32(np.zeros((batch, Bk))), i32(np.zeros(batch)), i32(np.zeros(batch))
    for _ in range(rounds):
        seq = [p + e for p, e in zip(prompts, emitted)]
        root = i32([s[-1] for s in seq])
        pos = i32([len(s) - 1 for s in seq])
        dt.tree_build(x["block_logits"], x["markov_a"], x["markov_b"], root, x["n_budget"], x["lam"], k=w.k,
                      Nmax=Nmax, temp=0.0, out=tree, ws=ws)
        ix = torch.cat([root[:, None], tree.tokens], 1).long()
        q, kt, vt = dm["q"][ix].contiguous(), dm["k"][ix].contiguous(), dm["v"][ix].contiguous()
        out = torch.zeros_like(q)
        dt.tree_verify_attn_paged(q, cache, dtable, pos, kt, vt, tree.anc, tree.n_nodes, scale, out, ws,
                                  depths=tree.depths, window=window, n_sink=sink)
        logits = (out.view(batch, Nmax + 1, -1).float() @ dm["w"].float())
        hist = i32(np.concatenate(seq))
        dt.logits_process(logits, logits, ws, tokens=tree.tokens, anc=tree.anc, n_nodes=tree.n_nodes,
                          history=hist, history_start=i32(np.concatenate([[0], np.cumsum([len(s) for s in seq])])),
                          n_prompt=i32([len(p) for p in prompts]), repetition=rho, presence=pres, frequency=freq)
        dt.tree_accept(logits, tree, Bk, 0.0, acc, n_acc, bonus, ws)
        dt.kv_commit(kt, vt, acc, n_acc, pos, cache, dtable, ws)
        assert dt.read_status(ws) == 0
        for b in range(batch):
            path = acc[b, : int(n_acc[b])].tolist()
            new = [int(tree.tokens[b, i]) for i in path] + [int(bonus[b])]
            first = len(seq[b]) - 1          # the root's position: this round's rows begin there
            for t in new:
                s = prompts[b] + emitted[b]
                o, mag = _reference(m, s, 1, code, window, sink, scale, tree_from=first)
                W = values(m["w"])
                z, _ = olog.process_row(o.reshape(-1) @ W, prompts[b], emitted[b], [], float(rho[b]),
                                        float(pres[b]), float(freq[b]))
                # the outputs' error bound through the projection, once for each of the two logits
                # compared (a penalty multiplies by at most 1.4), and fp32 sums of 256 products
                tol = 1.4 * 2 * (1.01 * 2.0 ** -7 + 256 * 2.0 ** -24) * ((np.abs(o) + mag).reshape(-1)
                                                                        @ np.abs(W)).max()
                assert z[t] >= z.max() - tol
                emitted[b].append(t)
    assert min(len(e) for e in emitted) >= rounds


def _reference(m, seq, n, code, window, sink, scale, tree_from=None):
    """fp64 attention outputs of the last n tokens of seq, and the weighted sums of |v|.  Cached
    rows are the quantised ones; rows from tree_from on are those of the round's own tree."""
    ix = torch.tensor(seq)
    kv = []
    for part in ("k", "v"):
        x = m[part][ix].float()
        c, s = to_codes(x, code)
        c = c.float() * s[..., None] if s is not None else c.float()
        if tree_from is not None:
            c[tree_from:] = x[tree_from:]
        kv.append(c.double().numpy())
    L = len(seq)
    ok = np.stack([oattn.seen_positions(L - n + i, L, window, sink) for i in range(n)])
    o, mag, _ = oattn.attend(values(m["q"][ix[L - n :]]), kv[0], kv[1], ok, scale)
    return o, mag
