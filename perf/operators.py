"""The serving-side operators of a draft-tree round, as cases that can be measured.

A decode round verifies a draft tree against a key/value cache and draws the next tokens from the
target's logits.  These operators bring that cache and those logits into the form the round needs:

  write   keys and values of new tokens (a prompt's chunk, or a round's accepted tree rows) quantised
          as they enter a paged cache
  read    cached rows gathered and dequantised into the packed prefix of the tree attention
  attn    attention of a chunk of new tokens over the paged cache (causal; optionally a sliding
          window with a few first tokens that stay visible)
  verify  the tree-masked attention of a round over the paged cache
  logits  penalties for repeated tokens, biases and grammar masks on the target's logits, for every
          node of a tree along its own path, or for single rows

`own` False computes the operators from elementary torch operations, True calls the library.
Shapes (lengths, trees) follow from the case alone; values from the seed.
"""
import math

import numpy as np
import torch

own = False

CODES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8, "f32": torch.float32}
TOP = {"e4m3": 448.0, "i8": 127.0}   # largest code of a quantised cache
TINY = 2.0 ** -100                   # rows whose largest value is below are scaled by it


def listed():
    return [
        # a batch of prompts enters an fp8 cache; k and v are slices of a fused projection's output
        dict(name="write_prefill_e4m3", op="write", code="e4m3", src="bf16", batch=16, rows=2048, hkv=8, d=128,
             page=64, fused=32, before=1024, shape=1),
        # the accepted rows of 64 trees are committed to an int8 cache
        dict(name="commit_batch_i8", op="commit", code="i8", src="bf16", batch=64, nmax=32, bk=7, hkv=8, d=128,
             page=16, before=8192, shape=2),
        # the prefixes of a load-adaptive batch of 64 (lognormal, 512 to 8192) are unpacked for another reader
        dict(name="read_batch_i8", op="read", code="i8", dst="bf16", batch=64, kv_lo=512, kv_hi=8192, hkv=8, d=128,
             page=32, shape=3),
        # one request's 2048-token prefix
        dict(name="read_one_e4m3", op="read", code="e4m3", dst="bf16", batch=1, kv_lo=2048, kv_hi=2048, hkv=8, d=128,
             page=128, shape=4),
        # the smallest step: one token, a 33-token cache, 2 query and 2 kv heads of 64
        dict(name="attn_tiny_bf16", op="attn", code="bf16", batch=1, rows_lo=1, rows_hi=1, kv_lo=33, kv_hi=33, hq=2,
             hkv=2, d=64, page=16, window=0, sink=0, shape=5),
        # single-token decoding of 64 requests, prefixes from 512 to 65536 tokens, fp8 cache
        dict(name="attn_decode_e4m3", op="attn", code="e4m3", batch=64, rows_lo=1, rows_hi=1, kv_lo=512, kv_hi=65536,
             hq=32, hkv=8, d=128, page=64, window=0, sink=0, shape=6),
        # three prompts' chunks of up to 2048 tokens over up to 8192 cached ones, bf16 cache
        dict(name="attn_chunk_bf16", op="attn", code="bf16", batch=3, rows_lo=1500, rows_hi=2048, kv_lo=4096,
             kv_hi=8192, hq=32, hkv=8, d=128, page=64, window=0, sink=0, shape=7),
        # two long prompts' chunks with a 4096-token window and 4 first tokens kept, int8 cache
        dict(name="attn_chunk_window_i8", op="attn", code="i8", batch=2, rows_lo=2048, rows_hi=4096, kv_lo=16384,
             kv_hi=32768, hq=32, hkv=8, d=128, page=128, window=4096, sink=4, shape=8),
        # one request's tree of 64 nodes over 4096 cached tokens
        dict(name="verify_one_bf16", op="verify", code="bf16", batch=1, nmax=64, kv_lo=4096, kv_hi=4096, hq=32, hkv=8,
             d=128, page=64, window=0, sink=0, shape=9),
        # a load-adaptive batch: 64 trees of up to 32 nodes, prefixes from 512 to 8192, fp8 cache
        dict(name="verify_batch_e4m3", op="verify", code="e4m3", batch=64, nmax=32, kv_lo=512, kv_hi=8192, hq=32,
             hkv=8, d=128, page=64, window=0, sink=0, shape=10),
        # the target rows of 16 trees with penalties along each path, biases and a mask per node
        dict(name="logits_tree_bf16", op="logits", code="bf16", batch=16, nmax=32, vocab=151936, hist_lo=256,
             hist_hi=8192, bias=64, mask=True, shape=11),
        # one row for each of 8 requests, no tree and no mask
        dict(name="logits_decode_f32", op="logits", code="f32", batch=8, nmax=0, vocab=151936, hist_lo=64,
             hist_hi=2048, bias=8, mask=False, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "commit", "read", "attn", "attn", "decode", "verify", "verify", "logits", "logits"])
    hkv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128])
    c = dict(op=op, shape=rng.randrange(1 << 30), hkv=hkv, d=d, page=rng.choice([16, 32, 64, 128]),
             code=rng.choice(["bf16", "e4m3", "i8"]))
    if op == "write":
        c.update(src=rng.choice(["bf16", "f32"]), batch=_log(rng, 1, 32), rows=_log(rng, 1, 1024),
                 fused=rng.choice([0, hkv * group]), before=_log(rng, 1, 4096))
    elif op == "commit":
        c.update(src=rng.choice(["bf16", "f32"]), batch=_log(rng, 1, 64), nmax=rng.randint(1, 64),
                 bk=rng.randint(1, 16), before=_log(rng, 1, 8192))
    elif op == "read":
        hi = _log(rng, 1, 8192)
        c.update(dst=rng.choice(["bf16", "f32"]), batch=_log(rng, 1, max(1, min(64, (1 << 16) // hi))),
                 kv_lo=_log(rng, 1, hi), kv_hi=hi)
    elif op in ("attn", "decode"):
        window = rng.choice([0, 0, _log(rng, 64, 4096)])
        if op == "decode":
            rows, hi = rng.choice([1, 1, 2, 5]), _log(rng, 8, 65536)
            c.update(batch=_log(rng, 1, max(1, min(64, (1 << 18) // hi))))
        else:
            rows = _log(rng, 8, 2048)
            hi = rows + _log(rng, 1, 8192)
            group = min(group, max(1, (1 << 29) // (rows * hi * hkv)))
            c.update(batch=_log(rng, 1, max(1, min(32, (1 << 29) // (rows * hi * hkv * group)))))
        c.update(op="attn", rows_lo=_log(rng, 1, rows), rows_hi=rows, kv_lo=max(1, hi // 4), kv_hi=hi, hq=hkv * group,
                 window=window, sink=rng.choice([0, 1, 4, 17]) if window else 0)
    elif op == "verify":
        hi, window = _log(rng, 1, 8192), rng.choice([0, 0, _log(rng, 128, 4096)])
        c.update(batch=_log(rng, 1, max(1, min(64, (1 << 17) // hi))), nmax=rng.randint(1, 64),
                 kv_lo=max(1, hi // 8), kv_hi=hi, hq=hkv * group, window=window, sink=rng.choice([0, 4]) if window else 0)
    else:
        nmax = rng.choice([0, rng.randint(1, 64)])
        vocab = _log(rng, 512, 151936)
        hi = _log(rng, 1, 8192)
        c = dict(op=op, shape=c["shape"], code=rng.choice(["bf16", "f32"]), nmax=nmax, vocab=vocab,
                 batch=_log(rng, 1, max(1, min(64, (1 << 26) // (vocab * (nmax + 1))))),
                 hist_lo=max(1, hi // 16), hist_hi=hi, bias=rng.choice([0, 1, 40]), mask=rng.random() < 0.5)
    return c


# --------------------------------------------------------------- shapes --
def _lognormal(r, n, lo, hi):
    """Lengths as the load-adaptive batch draws them, spread over [lo, hi]; the last is the longest."""
    if lo >= hi:
        return np.full(n, hi, np.int64)
    got = np.clip(np.round(2 * lo * np.exp(0.9 * r.standard_normal(n))), lo, hi).astype(np.int64)
    got[-1] = hi
    return got


def _trees(r, batch, nmax):
    """Node counts and parents (-1 = the root) of ragged random trees."""
    n = r.integers(max(1, nmax // 4), nmax + 1, batch) if nmax else np.zeros(batch, np.int64)
    if nmax:
        n[-1] = nmax
    parent = np.full((batch, max(nmax, 1)), -1, np.int64)
    depth = np.ones((batch, max(nmax, 1)), np.int64)
    anc = np.zeros((batch, max(nmax, 1)), np.uint64)
    for b in range(batch):
        for i in range(n[b]):
            p = int(r.integers(-1, i)) if i else -1
            while p >= 0 and depth[b, p] >= 16:
                p = parent[b, p]
            parent[b, i] = p
            depth[b, i] = 1 if p < 0 else depth[b, p] + 1
            anc[b, i] = np.uint64(1 << i) | (anc[b, p] if p >= 0 else np.uint64(0))
    return n, parent, depth, anc


def _shapes(case):
    """Every length that a case has, from the case alone."""
    r = np.random.default_rng([case["shape"], 17])
    op, batch = case["op"], case["batch"]
    s = {}
    if op == "write":
        s["rows"] = r.integers(max(1, case["rows"] // 2), case["rows"] + 1, batch)
        s["rows"][-1] = case["rows"]
        s["pos"] = r.integers(0, case["before"] + 1, batch)
        s["kv"] = s["pos"] + s["rows"]
    elif op == "commit":
        s["n"], s["parent"], s["depth"], s["anc"] = _trees(r, batch, case["nmax"])
        acc = np.full((batch, case["bk"]), -1, np.int64)
        n_acc = np.zeros(batch, np.int64)
        for b in range(batch):
            i = int(r.integers(-1, s["n"][b]))
            path = []
            while i >= 0:
                path.append(i)
                i = int(s["parent"][b, i])
            path = path[::-1][:case["bk"]]
            acc[b, :len(path)], n_acc[b] = path, len(path)
        s["acc"], s["n_acc"] = acc, n_acc
        s["rows"] = n_acc + 1
        s["pos"] = _lognormal(r, batch, max(1, case["before"] // 16), case["before"])
        s["kv"] = s["pos"] + s["rows"]
    elif op == "read":
        s["kv"] = _lognormal(r, batch, case["kv_lo"], case["kv_hi"])
    elif op == "attn":
        s["kv"] = _lognormal(r, batch, case["kv_lo"], case["kv_hi"])
        s["rows"] = np.minimum(r.integers(case["rows_lo"], case["rows_hi"] + 1, batch), s["kv"])
    elif op == "verify":
        s["kv"] = _lognormal(r, batch, case["kv_lo"], case["kv_hi"])
        s["n"], s["parent"], s["depth"], s["anc"] = _trees(r, batch, case["nmax"])
    else:
        s["n"], s["parent"], s["depth"], s["anc"] = _trees(r, batch, case["nmax"])
        s["hist"] = _lognormal(r, batch, case["hist_lo"], case["hist_hi"])
        s["prompt"] = s["hist"] // 2
    return s


def _pairs(case, s):
    """How many (row, cached position) pairs are visible."""
    total = 0
    w, sink = case["window"], case["sink"]
    for b in range(case["batch"]):
        kv = int(s["kv"][b])
        if case["op"] == "attn":
            p = np.arange(kv - int(s["rows"][b]), kv)
            last = p + 1
        else:
            p = kv + np.concatenate([[0], s["depth"][b, :s["n"][b]]])
            last = np.full(len(p), kv)
        first = np.maximum(0, p - w + 1) if w else np.zeros_like(p)
        total += int(np.sum(last - np.minimum(first, last)) + np.sum(np.minimum(np.minimum(first, sink), last)))
    return total


def _reach(case, s, b):
    """How many cached positions any row of request b sees."""
    kv, w = int(s["kv"][b]), case["window"]
    if not w:
        return kv
    low = kv - int(s["rows"][b]) if case["op"] == "attn" else kv
    first = max(0, low - w + 1)
    return kv - min(first, kv) + min(first, case["sink"], kv)


def work(case):
    s, op, batch = _shapes(case), case["op"], case["batch"]
    size = {"bf16": 2, "f32": 4, "e4m3": 1, "i8": 1}
    if op in ("write", "commit", "read"):
        n = int(np.sum(s["kv"] if op == "read" else s["rows"]))
        vals = 2 * n * case["hkv"] * case["d"]
        scales = 2 * n * case["hkv"] * 4 if case["code"] in TOP else 0
        other = case["dst"] if op == "read" else case["src"]
        return {"bytes": vals * (size[case["code"]] + size[other]) + scales, "flops": 4 * vals if scales else 0}
    if op in ("attn", "verify"):
        row = case["hkv"] * (2 * case["d"] * size[case["code"]] + (8 if case["code"] in TOP else 0))
        nbytes = sum(_reach(case, s, b) for b in range(batch)) * row
        pairs = _pairs(case, s)
        if op == "attn":
            rows = int(np.sum(s["rows"]))
        else:
            rows = int(np.sum(s["n"] + 1))
            nbytes += rows * case["hkv"] * 2 * case["d"] * 2
            pairs += int(sum(1 + np.sum(1 + s["depth"][b, :s["n"][b]]) for b in range(batch)))
        nbytes += rows * case["hq"] * case["d"] * 2 * 2
        return {"bytes": nbytes, "flops": 4 * pairs * case["hq"] * case["d"]}
    rows = int(np.sum(s["n"] + 1))
    nbytes = rows * case["vocab"] * size[case["code"]] * 2 + int(np.sum(s["hist"])) * 4 + batch * case["bias"] * 8
    if case["mask"]:
        nbytes += rows * ((case["vocab"] + 31) // 32) * 4
    return {"bytes": nbytes, "flops": 4 * rows * case["vocab"]}


# -------------------------------------------------------------- inputs --
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 11)


def _ints(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(torch.int32).cuda()


def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _cache(case, s, g):
    """A pool with spare pages, its pages dealt out in random order, filled with cached rows."""
    need = -(-s["kv"] // case["page"])
    pool = int(np.sum(need)) + 3
    order = np.random.default_rng([case["shape"], 23]).permutation(pool)
    table = np.zeros((case["batch"], int(need.max())), np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    c = {"table": _ints(table)}
    shape = (pool, case["hkv"], case["page"], case["d"])
    for part in ("k", "v"):
        if case["code"] == "bf16":
            c[part] = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        else:  # codes as quantised normal rows have them: the largest is the top, the scale about 3.3 / top
            x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
            x.mul_(TOP[case["code"]] / 3.3).clamp_(-TOP[case["code"]], TOP[case["code"]])
            c[part] = x.round_().to(torch.int8) if case["code"] == "i8" else x.to(torch.float8_e4m3fn)
            del x
            scale = torch.empty(shape[:3], device="cuda").uniform_(0.8, 1.2, generator=g)
            c[part + "_scale"] = scale * (3.3 / TOP[case["code"]])
    return c


def _tree_tensors(s):
    return dict(n_nodes=_ints(s["n"]), depths=_ints(s["depth"]),
                anc=torch.as_tensor(s["anc"].view(np.int64)).cuda())


def prepare(case, seed):
    g, s, op, batch = _gen(seed), _shapes(case), case["op"], case["batch"]
    st = {"case": dict(case), "op": op}
    normal = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)
    if op != "logits":
        st.update(_cache(case, s, g))
        hkv, d = case["hkv"], case["d"]
    if op == "write":
        total = int(np.sum(s["rows"]))
        heads = case["fused"] + 2 * hkv
        qkv = normal((total, heads, d), CODES[case["src"]])
        st.update(new_k=qkv[:, case["fused"]:case["fused"] + hkv], new_v=qkv[:, case["fused"] + hkv:],
                  row_start=_ints(_starts(s["rows"])), pos=_ints(s["pos"]))
    elif op == "commit":
        st.update(new_k=normal((batch, case["nmax"] + 1, hkv, d), CODES[case["src"]]),
                  new_v=normal((batch, case["nmax"] + 1, hkv, d), CODES[case["src"]]),
                  acc=_ints(s["acc"]), n_acc=_ints(s["n_acc"]), pos=_ints(s["pos"]))
    elif op == "read":
        total = int(np.sum(s["kv"]))
        st.update(row_start=_ints(_starts(s["kv"])), pos=_ints(np.zeros(batch)), most=int(s["kv"].max()), total=total,
                  out_k=torch.zeros((total, hkv, d), dtype=CODES[case["dst"]], device="cuda"),
                  out_v=torch.zeros((total, hkv, d), dtype=CODES[case["dst"]], device="cuda"))
    elif op == "attn":
        total = int(np.sum(s["rows"]))
        st.update(q=normal((total, case["hq"], d), torch.bfloat16), row_start=_ints(_starts(s["rows"])),
                  kv_len=_ints(s["kv"]), most=int(s["kv"].max()), most_rows=case["rows_hi"], scale=d ** -0.5)
        st["out"] = torch.zeros_like(st["q"])
    elif op == "verify":
        rows = case["nmax"] + 1
        st.update(q=normal((batch, rows, case["hq"], d), torch.bfloat16), prefix_len=_ints(s["kv"]),
                  k_tree=normal((batch, rows, hkv, d), torch.bfloat16), most=int(s["kv"].max()), scale=d ** -0.5,
                  v_tree=normal((batch, rows, hkv, d), torch.bfloat16), **_tree_tensors(s))
        st["out"] = torch.zeros_like(st["q"])
    else:
        V, rows = case["vocab"], case["nmax"] + 1
        logits = normal((batch, rows, V), torch.float32).mul_(3.0).to(CODES[case["code"]])
        # tokens of a text repeat: half of them come from a few hundred common ones
        def tokens(shape):
            wide = torch.randint(0, V, shape, device="cuda", generator=g)
            near = torch.randint(0, min(V, 300), shape, device="cuda", generator=g)
            return torch.where(torch.rand(shape, device="cuda", generator=g) < 0.5, near, wide).to(torch.int32)
        uni = lambda lo, hi: torch.empty(batch, device="cuda").uniform_(lo, hi, generator=g)
        st.update(logits=logits, out=torch.zeros_like(logits), history=tokens((int(np.sum(s["hist"])),)),
                  hist_start=_ints(_starts(s["hist"])), n_prompt=_ints(s["prompt"]), most_hist=int(s["hist"].max()),
                  rep=uni(1.0, 1.3), pres=uni(0.0, 0.8), freq=uni(0.0, 0.4), **_tree_tensors(s))
        st["tokens"] = tokens((batch, max(case["nmax"], 1)))
        if case["bias"]:
            k = min(case["bias"], V)
            order = torch.rand((batch, V), device="cuda", generator=g)
            st["bias_token"] = order.topk(k, 1).indices.to(torch.int32).reshape(-1)
            st["bias_value"] = normal((batch * k,), torch.float32).mul_(4.0)
            st["bias_start"] = _ints(np.arange(batch + 1) * k)
        if case["mask"]:
            # grammar states: half of them let a few tokens through, half of them most
            W = (V + 31) // 32
            word = lambda: torch.randint(-2 ** 31, 2 ** 31, (batch * rows, W), device="cuda", generator=g)
            few, most = word() & word() & word() & word() & word(), word() | word() | word() | word()
            pick = torch.rand((batch * rows, 1), device="cuda", generator=g) < 0.5
            st["mask"] = torch.where(pick, few, most).to(torch.int32)
            state = torch.randperm(batch * rows, device="cuda", generator=g)
            st["mask_row"] = state.to(torch.int32).reshape(batch, rows)
    return st


# ---------------------------------------------------------- plain forms --
def _rows_of(start, most):
    """[batch, most] packed row of each request's i-th row, and which of them there are."""
    i = torch.arange(most, device="cuda")
    n = start[1:] - start[:-1]
    there = i[None] < n[:, None]
    return torch.where(there, start[:-1, None] + i[None], 0).long(), there


def _gathered(st, part, pos):
    """float32 rows [batch, L, Hkv, d] of the cached positions pos [batch, L]."""
    page = st["case"]["page"]
    p = torch.gather(st["table"].long(), 1, pos // page)
    x = st[part][p, :, pos % page].float()
    if part + "_scale" in st:
        x = x * st[part + "_scale"][p, :, pos % page][..., None]
    return x


def _quantised(x, code):
    """The codes and scales of float32 rows [..., d]."""
    if code == "bf16":
        return x.to(torch.bfloat16), None
    top = x.abs().amax(-1, keepdim=True).clamp_min(TINY)
    most = torch.full_like(top, TOP[code])   # a tensor: a quotient with a number would be a product with its inverse
    q = x * (most / top)
    q = q.round().clamp(-127, 127).to(torch.int8) if code == "i8" else q.clamp(-448, 448).to(torch.float8_e4m3fn)
    return q, (top / most)[..., 0]


def _plain_write(st):
    case = st["case"]
    if st["op"] == "write":
        total = st["new_k"].shape[0]
        src = torch.arange(total, device="cuda")
        b = torch.searchsorted(st["row_start"], src.int(), right=True) - 1
        pos = (st["pos"][b] + src - st["row_start"][b]).long()
        k, v = st["new_k"], st["new_v"]
    else:
        rows, bk = case["nmax"] + 1, case["bk"]
        i = torch.arange(bk + 1, device="cuda")[None].expand(case["batch"], -1)
        b = torch.arange(case["batch"], device="cuda")[:, None].expand_as(i)
        there = i <= st["n_acc"][:, None]
        path = torch.cat([torch.zeros_like(st["acc"][:, :1]), st["acc"] + 1], 1)
        src = (b * rows + path)[there].long()
        pos, b = (st["pos"][:, None] + i)[there].long(), b[there]
        k, v = st["new_k"].flatten(0, 1)[src], st["new_v"].flatten(0, 1)[src]
    page = st["table"][b, pos // case["page"]].long()
    slot = pos % case["page"]
    got = []
    for part, x in (("k", k), ("v", v)):
        q, scale = _quantised(x.float(), case["code"])
        pool = st[part].view(torch.int8) if case["code"] != "bf16" else st[part]
        pool[page, :, slot] = q.view(pool.dtype)
        got.append(st[part])
        if scale is not None:
            st[part + "_scale"][page, :, slot] = scale
            got.append(st[part + "_scale"])
    return got


def _plain_read(st):
    dst = CODES[st["case"]["dst"]]
    _, there = _rows_of(st["row_start"], st["most"])
    pos = torch.arange(st["most"], device="cuda")[None].expand(there.shape[0], -1)
    pos = torch.where(there, pos, 0)
    st["out_k"].copy_(_gathered(st, "k", pos)[there].to(dst))
    st["out_v"].copy_(_gathered(st, "v", pos)[there].to(dst))
    return [st["out_k"], st["out_v"]]


def _softmaxed(q, k, v, seen, scale):
    """q [b, R, Hq, d], k/v [b, L, Hkv, d], seen [b, R, L] -> [b, R, Hq, d]; rows that see nothing are 0."""
    B, R, Hq, d = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    q = q.reshape(B, R, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * R, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(scale).view(B, Hkv, G, R, -1)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, G * R, -1), v.permute(0, 2, 1, 3)).view(B, Hkv, G, R, d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, R, Hq, d)


def _window(case, pos, at):
    """Which positions `at` the rows at `pos` may see by the window and the first tokens."""
    if not case["window"]:
        return torch.ones_like(at <= pos)
    return (at > pos - case["window"]) | (at < case["sink"])


def _plain_attn(st):
    case = st["case"]
    src, there = _rows_of(st["row_start"], st["most_rows"])
    n = (st["row_start"][1:] - st["row_start"][:-1])[:, None]
    pos = st["kv_len"][:, None] - n + torch.arange(st["most_rows"], device="cuda")[None]
    at = torch.arange(st["most"], device="cuda")
    cached = torch.where(at[None] < st["kv_len"][:, None], at[None], 0).long()
    seen = (at[None, None] <= pos[..., None]) & _window(case, pos[..., None], at[None, None])
    o = _softmaxed(st["q"][src].float(), _gathered(st, "k", cached), _gathered(st, "v", cached), seen, st["scale"])
    st["out"][src[there]] = o[there].to(torch.bfloat16)
    return st["out"]


def _bits(anc, n):
    return ((anc[..., None] >> torch.arange(n, device="cuda")) & 1).bool()


def _plain_verify(st):
    case = st["case"]
    rows = case["nmax"] + 1
    i = torch.arange(rows, device="cuda")
    there = i[None] <= st["n_nodes"][:, None]
    at = torch.arange(st["most"], device="cuda")
    kept = at[None] < st["prefix_len"][:, None]
    cached = torch.where(kept, at[None], 0).long()
    pos = st["prefix_len"][:, None] + torch.cat([torch.zeros_like(st["depths"][:, :1]), st["depths"]], 1)
    seen = kept[:, None] & _window(case, pos[..., None], at[None, None])
    tree = torch.zeros((case["batch"], rows, rows), dtype=torch.bool, device="cuda")
    tree[:, :, 0] = True
    tree[:, 1:, 1:] = _bits(st["anc"], case["nmax"])
    k = torch.cat([_gathered(st, "k", cached), st["k_tree"].float()], 1)
    v = torch.cat([_gathered(st, "v", cached), st["v_tree"].float()], 1)
    o = _softmaxed(st["q"].float(), k, v, torch.cat([seen, tree], 2), st["scale"])
    st["out"].copy_(torch.where(there[..., None, None], o.to(torch.bfloat16), st["out"]))
    return st["out"]


def _plain_logits(st):
    case = st["case"]
    batch, V, rows = case["batch"], case["vocab"], case["nmax"] + 1
    src, there = _rows_of(st["hist_start"], st["most_hist"])
    tok = torch.where(there, st["history"][src].long(), 0)
    of_prompt = torch.arange(st["most_hist"], device="cuda")[None] < st["n_prompt"][:, None]
    counts = lambda w: torch.zeros((batch, V), dtype=torch.int32, device="cuda").scatter_add_(1, tok, w.int())
    prompt, made = counts(there & of_prompt)[:, None], counts(there & ~of_prompt)[:, None]
    if case["nmax"]:
        on = torch.zeros((batch, rows, case["nmax"]), dtype=torch.int32, device="cuda")
        on[:, 1:] = _bits(st["anc"], case["nmax"])
        path = torch.zeros((batch, rows, V), dtype=torch.int32, device="cuda")
        path.scatter_add_(2, st["tokens"].long()[:, None].expand(-1, rows, -1), on)
        made = made + path
    x = st["logits"].float()
    per = lambda a: a[:, None, None]
    x = torch.where((prompt + made) > 0, torch.where(x > 0, x / per(st["rep"]), x * per(st["rep"])), x)
    x = x - per(st["freq"]) * made - torch.where(made > 0, per(st["pres"]), 0.0)
    if case["bias"]:
        add = torch.zeros((batch, V), device="cuda")
        add.scatter_(1, st["bias_token"].long().view(batch, -1), st["bias_value"].view(batch, -1))
        x = x + add[:, None]
    if case["mask"]:
        bit = torch.arange(32, device="cuda", dtype=torch.int32)
        ok = ((st["mask"][st["mask_row"].long()][..., None] >> bit) & 1).bool().flatten(2)[..., :V]
        x = torch.where(ok, x, -math.inf)
    live = (torch.arange(rows, device="cuda")[None] <= st["n_nodes"][:, None])[..., None]
    st["out"].copy_(torch.where(live, x.to(st["out"].dtype), st["out"]))
    return st["out"]


# --------------------------------------------------------- own operators --
def _own(st):
    import draft_tree_construction_markov_b200 as dt
    case, op = st["case"], st["op"]
    if op != "logits" and "cache" not in st:
        st["cache"] = dt.KVCache(st["k"], st["v"], st.get("k_scale"), st.get("v_scale"))
    if "ws" not in st:
        if op == "attn":
            need = dt.paged_attn_workspace_bytes(case["batch"], st["q"].shape[0], case["hq"], case["hkv"], case["d"])
        elif op == "verify":
            need = dt.verify_paged_workspace_bytes(case["batch"], case["nmax"], case["hq"], case["hkv"], case["d"])
        elif op == "logits":
            need = dt.logits_workspace_bytes()
        else:
            need = dt.kv_workspace_bytes()
        st["ws"] = dt.workspace(need)
    if op in ("write", "commit"):
        if op == "write":
            dt.kv_write(st["new_k"], st["new_v"], st["row_start"], st["pos"], st["cache"], st["table"], st["ws"])
        else:
            dt.kv_commit(st["new_k"], st["new_v"], st["acc"], st["n_acc"], st["pos"], st["cache"], st["table"],
                         st["ws"])
        return [st[x] for x in ("k", "k_scale", "v", "v_scale") if x in st]
    if op == "read":
        dt.kv_read(st["cache"], st["table"], st["row_start"], st["pos"], st["out_k"], st["out_v"], st["ws"])
        return [st["out_k"], st["out_v"]]
    if op == "attn":
        return dt.paged_attn(st["q"], st["row_start"], st["cache"], st["table"], st["kv_len"], st["scale"], st["out"],
                             st["ws"], max_rows=st["most_rows"], window=case["window"], n_sink=case["sink"])
    if op == "verify":
        return dt.tree_verify_attn_paged(st["q"], st["cache"], st["table"], st["prefix_len"], st["k_tree"],
                                         st["v_tree"], st["anc"], st["n_nodes"], st["scale"], st["out"],
                                         st["ws"], depths=st["depths"], window=case["window"], n_sink=case["sink"])
    tree = {}
    if case["nmax"]:
        tree = dict(tokens=st["tokens"], anc=st["anc"], n_nodes=st["n_nodes"])
    return dt.logits_process(st["logits"], st["out"], st["ws"], history=st["history"], history_start=st["hist_start"],
                             n_prompt=st["n_prompt"], repetition=st["rep"], presence=st["pres"], frequency=st["freq"],
                             bias_start=st.get("bias_start"), bias_token=st.get("bias_token"),
                             bias_value=st.get("bias_value"), mask=st.get("mask"),
                             mask_row=st.get("mask_row"), **tree)


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "commit": _plain_write, "read": _plain_read, "attn": _plain_attn,
            "verify": _plain_verify, "logits": _plain_logits}[state["op"]](state)


# --------------------------------------------------- from the definition --
def _e4m3(x):
    """float64 values rounded to the nearest of sign, 4 exponent and 3 mantissa bits, ties to even."""
    exp = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -9))).clamp_min(-6.0)
    step = torch.exp2(exp - 3.0)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_rows(st, part, b, n):
    """float64 rows [n, Hkv, d] of request b's first n positions."""
    page = st["case"]["page"]
    pages = st["table"][b, :-(-n // page)].long()
    x = st[part][pages].double()
    if part + "_scale" in st:
        x = x * st[part + "_scale"][pages].double()[..., None]
    return x.transpose(1, 2).reshape(-1, *x.shape[1::2])[:n]


def _exact_heads(q, k, v, seen, scale):
    """q [R, Hq, d], k/v [L, Hkv, d], seen [R, L] -> [R, Hq, d], head by head."""
    out = torch.zeros_like(q)
    G = q.shape[1] // k.shape[1]
    blank = ~seen.any(1)
    for h in range(q.shape[1]):
        x = (q[:, h] @ k[:, h // G].T * scale).masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(x, 1, keepdim=True)
        out[:, h] = torch.exp(x - lse).masked_fill(blank[:, None], 0.0) @ v[:, h // G]
    return out


def exact(case, seed):
    s, op = _shapes(case), case["op"]
    st = prepare(case, seed)
    if op in ("write", "commit"):
        code, got = case["code"], []
        for part in ("k", "v"):
            pool = st[part].double()
            scales = st[part + "_scale"].double() if code in TOP else None
            for b in range(case["batch"]):
                n = int(s["rows"][b])
                pos = int(s["pos"][b]) + torch.arange(n, device="cuda")
                page = st["table"][b, pos // case["page"]].long()
                if op == "write":
                    at = int(st["row_start"][b])
                    x = st["new_" + part][at:at + n].double()
                else:
                    x = st["new_" + part][b, [0] + [int(i) + 1 for i in s["acc"][b, :n - 1]]].double()
                if code in TOP:
                    top = x.abs().amax(2).clamp_min(TINY)
                    x = x * (TOP[code] / top)[..., None]
                    scales[page, :, pos % case["page"]] = top / TOP[code]
                    x = _e4m3(x) if code == "e4m3" else torch.round(x)
                pool[page, :, pos % case["page"]] = x
            got += [None if code == "i8" else pool] + ([scales] if code in TOP else [])
        return got
    if op == "read":
        rows = lambda part: [_exact_rows(st, part, b, int(s["kv"][b])) for b in range(case["batch"])]
        return [torch.cat(rows("k")), torch.cat(rows("v"))]
    if op in ("attn", "verify"):
        out = st["out"].double()
        for b in range(case["batch"]):
            kv = int(s["kv"][b])
            k, v = (_exact_rows(st, part, b, kv) for part in ("k", "v"))
            at = torch.arange(kv, device="cuda")
            if op == "attn":
                a = int(st["row_start"][b])
                z = int(st["row_start"][b + 1])
                pos = torch.arange(kv - (z - a), kv, device="cuda")
                q = st["q"][a:z].double()
            else:
                n = int(s["n"][b]) + 1
                pos = kv + torch.as_tensor(np.concatenate([[0], s["depth"][b, :n - 1]])).cuda()
                q = st["q"][b, :n].double()
            seen = at[None] <= pos[:, None]
            if case["window"]:
                seen &= (pos[:, None] - at[None] < case["window"]) | (at[None] < case["sink"])
            if op == "verify":
                own_rows = torch.zeros((n, n), dtype=torch.bool)
                for i in range(n):
                    own_rows[i, 0] = True
                    j = i - 1
                    while j >= 0:
                        own_rows[i, j + 1] = True
                        j = int(s["parent"][b, j])
                seen = torch.cat([seen, own_rows.cuda()], 1)
                k, v = torch.cat([k, st["k_tree"][b, :n].double()]), torch.cat([v, st["v_tree"][b, :n].double()])
            o = _exact_heads(q, k, v, seen, st["scale"])
            if op == "attn":
                out[a:z] = o
            else:
                out[b, :n] = o
        return out
    out = st["out"].double()
    V = case["vocab"]
    for b in range(case["batch"]):
        a, z = int(st["hist_start"][b]), int(st["hist_start"][b + 1])
        past = st["history"][a:z].long()
        prompt = torch.bincount(past[:int(s["prompt"][b])], minlength=V)
        made0 = torch.bincount(past[int(s["prompt"][b]):], minlength=V)
        rep, pres, freq = (float(st[x][b]) for x in ("rep", "pres", "freq"))
        for i in range(int(s["n"][b]) + 1):
            made, j = made0.clone(), i - 1
            while j >= 0:
                made[int(st["tokens"][b, j])] += 1
                j = int(s["parent"][b, j])
            x = st["logits"][b, i].double()
            again = (prompt + made) > 0
            x = torch.where(again & (x > 0), x / rep, torch.where(again, x * rep, x))
            x = x - freq * made - pres * (made > 0)
            if case["bias"]:
                y, w = int(st["bias_start"][b]), int(st["bias_start"][b + 1])
                x[st["bias_token"][y:w].long()] += st["bias_value"][y:w].double()
            if case["mask"]:
                word = st["mask"][int(st["mask_row"][b, i])].cpu().numpy().view(np.uint8)
                ok = np.unpackbits(word, bitorder="little")[:V].astype(bool)
                x[~torch.as_tensor(ok).cuda()] = -math.inf
            out[b, i] = x
    return out
