"""The serving operators together in fp32, where rounding is small enough to tell tokens apart.

The target of tests/test_gpu_serving_round.py with fp32 rows, queries and cache.  Greedy acceptance is
lossless, so a round has to emit what step-by-step decoding in fp64 emits, token for token; the drafts
are that continuation, so that rounds accept whole paths and the penalties along them decide.  The
operators' error is bounded by 0.007 of a logit, and the best two logits of every step are further
apart.  That the comparison notices a penalty left out, a path not counted or a prompt counted as
generated is shown by the oracle making these mistakes.
"""
import numpy as np
import pytest
import torch

from gen import make_workload
from oracle import logits as olog
from oracle import paged_attn as oattn
from tests.serving_util import page_table, values

if torch.cuda.is_available():
    import draft_tree_construction_markov_b200 as dt
    from tests.gpu_util import build_inputs
    from tests.serving_util import cuda

HQ, HKV, D, V, ROUNDS, BK, NMAX = 4, 2, 64, 512, 4, 4, 8
SCALE = D ** -0.5
PROMPTS = (40, 7, 23)


def _target(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    E = r(V, 64)
    return dict(q=(E @ r(64, HQ * D) / 8).view(V, HQ, D), k=(E @ r(64, HKV * D) / 8).view(V, HKV, D),
                v=(E @ r(64, HKV * D) / 8).view(V, HKV, D), w=r(HQ * D, V) / 2)


def _settings():
    g = np.random.default_rng(1)
    prompts = [g.integers(0, V, n).tolist() for n in PROMPTS]
    par = [g.uniform(*r, len(prompts)).astype(np.float32) for r in ((1.1, 1.5), (0.5, 2.0), (0.3, 1.0))]
    return prompts, par


def _step(m64, seq, window, sink):
    """The last token's fp64 logits before the penalties, and what the fp32 operators may be off by:
    every score and weight by the bound of tests/test_gpu_paged_attn.py, the projection by a sum of
    HQ D products."""
    L = len(seq)
    ok = oattn.seen_positions(L - 1, L, window, sink)[None]
    o, mag, big = oattn.attend(m64["q"][seq[-1:]], m64["k"][seq], m64["v"][seq], ok, SCALE)
    rel = 2 * (D + 8) * 2.0 ** -24 * big[..., None] + 2 * (L + NMAX) * 2.0 ** -24 + 2.0 ** -20
    W = m64["w"]
    off = (rel * mag).reshape(-1) @ np.abs(W) + HQ * D * 2.0 ** -24 * (np.abs(o).reshape(-1) @ np.abs(W))
    return o.reshape(-1) @ W, off.max()


def _decode(m64, prompt, n, rho, pres, freq, window, sink, mistake=None):
    """n greedy tokens after the prompt, and the least distance of a step's best two logits over what
    they may be off by.  A mistake of the rounds' kind counts a round's own tokens (its path) wrongly."""
    out, least = [], np.inf
    for i in range(n):
        z, off = _step(m64, prompt + out, window, sink)
        made = out[: i - i % (BK + 1)] if mistake == "path" else out
        past, gen = ([], prompt + made) if mistake == "prompt" else (prompt, made)
        r, p, f = (1.0 if mistake == "rho" else rho, 0.0 if mistake == "pres" else pres,
                   0.0 if mistake == "freq" else freq)
        z, big = olog.process_row(z, past, gen, [], r, p, f)
        best = np.argsort(z)[-2:]
        least = min(least, (z[best[1]] - z[best[0]]) / (2 * (1.5 * off + 6 * 2.0 ** -24 * big.max())))
        out.append(int(best[1]))
    return out, least


def _m64(m):
    return {k: values(t) for k, t in m.items()}


@pytest.mark.parametrize("window,sink", [(0, 0), (24, 4)])
def test_the_steps_are_told_apart_and_mistakes_show(window, sink):
    """On the CPU: of the oracle alone."""
    m64, (prompts, par) = _m64(_target(307)), _settings()
    n = ROUNDS * (BK + 1)
    right = [_decode(m64, p, n, *(x[b] for x in par), window, sink) for b, p in enumerate(prompts)]
    assert min(least for _, least in right) > 1
    for mistake in ("path", "prompt", "rho", "pres", "freq"):
        wrong = [_decode(m64, p, n, *(x[b] for x in par), window, sink, mistake)[0] for b, p in enumerate(prompts)]
        assert wrong != [t for t, _ in right], mistake


@pytest.mark.gpu
@pytest.mark.parametrize("window,sink", [(0, 0), (24, 4)])
def test_rounds_in_fp32_emit_step_by_step_decoding_exactly(window, sink):
    w = make_workload("tiny", seed=3, batch=3, N=NMAX)
    assert (w.V, w.Bk, w.Nmax) == (V, BK, NMAX)
    m, (prompts, (rho, pres, freq)) = _target(307), _settings()
    m64, dm, batch = _m64(m), {k: t.cuda() for k, t in m.items()}, len(prompts)
    want = [_decode(m64, p, ROUNDS * (BK + 1), rho[b], pres[b], freq[b], window, sink)[0]
            for b, p in enumerate(prompts)]
    table, pool = page_table(np.random.default_rng(2), [len(p) + ROUNDS * (BK + 1) + 1 for p in prompts], 8)
    cache, table = dt.KVCache.empty(pool, 8, HKV, D, torch.float32), cuda(table)
    i32 = lambda a: cuda(np.asarray(a, np.int32))
    ws = dt.workspace(max(dt.kv_workspace_bytes(), dt.paged_attn_workspace_bytes(batch, 128, HQ, HKV, D),
                          dt.verify_paged_workspace_bytes(batch, NMAX, HQ, HKV, D),
                          dt.accept_workspace_bytes(batch, NMAX, V),
                          dt.build_workspace_bytes(batch, BK, V, w.r, w.k, NMAX)))
    ends = [len(p) - 1 for p in prompts]
    ix = torch.tensor([t for p in prompts for t in p[:-1]]).cuda()
    dt.kv_write(dm["k"][ix], dm["v"][ix], i32(np.concatenate([[0], np.cumsum(ends)])), i32([0] * batch), cache,
                table, ws)
    x = build_inputs(w)
    draft = x["block_logits"].clone()
    tree = dt.Tree.empty(batch, NMAX, V)
    acc, n_acc, bonus = i32(np.zeros((batch, BK))), i32(np.zeros(batch)), i32(np.zeros(batch))
    emitted, accepted = [[] for _ in prompts], 0
    for _ in range(ROUNDS):
        seq = [p + e for p, e in zip(prompts, emitted)]
        root, pos = i32([s[-1] for s in seq]), i32([len(s) - 1 for s in seq])
        draft.copy_(x["block_logits"])
        for b in range(batch):
            for i, t in enumerate(want[b][len(emitted[b]) :][:BK]):
                draft[b, i, t] = 30.0
        dt.tree_build(draft, x["markov_a"], x["markov_b"], root, x["n_budget"], x["lam"], k=w.k, Nmax=NMAX,
                      temp=0.0, out=tree, ws=ws)
        ix = torch.cat([root[:, None], tree.tokens], 1).long()
        q, kt, vt = dm["q"][ix].contiguous(), dm["k"][ix].contiguous(), dm["v"][ix].contiguous()
        out = torch.zeros_like(q)
        dt.tree_verify_attn_paged(q, cache, table, pos, kt, vt, tree.anc, tree.n_nodes, SCALE, out, ws,
                                  depths=tree.depths, window=window, n_sink=sink)
        # (the projection in fp64, rounded once: what it adds is within the bound)
        logits = (out.view(batch, NMAX + 1, -1).double() @ dm["w"].double()).float()
        dt.logits_process(logits, logits, ws, tokens=tree.tokens, anc=tree.anc, n_nodes=tree.n_nodes,
                          history=i32(np.concatenate(seq)),
                          history_start=i32(np.concatenate([[0], np.cumsum([len(s) for s in seq])])),
                          n_prompt=i32([len(p) for p in prompts]), repetition=cuda(rho), presence=cuda(pres),
                          frequency=cuda(freq))
        dt.tree_accept(logits, tree, BK, 0.0, acc, n_acc, bonus, ws)
        dt.kv_commit(kt, vt, acc, n_acc, pos, cache, table, ws)
        assert dt.read_status(ws) == 0
        for b in range(batch):
            path = acc[b, : int(n_acc[b])].tolist()
            emitted[b] += [int(tree.tokens[b, i]) for i in path] + [int(bonus[b])]
            accepted += len(path)
            assert emitted[b] == want[b][: len(emitted[b])]
    assert accepted >= batch * ROUNDS * (BK - 1)         # whole paths, so that paths were counted
