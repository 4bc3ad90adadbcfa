"""Shared by the tests of the paged cache, the attention over it and the logits processing."""
import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
          "i8": torch.int8}
TOP = {"e4m3": 448.0, "i8": 127.0}


def page_table(g, lens, page, spare=3):
    """A table of shuffled pages for requests of the given lengths, and the pool's size."""
    need = [-(-int(n) // page) for n in lens]
    order = g.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)  # unused entries: no page
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, len(order)


def to_codes(x, code):
    """float32 array -> CPU codes [..., d] and scales, by the fp32 definition."""
    t = torch.as_tensor(np.asarray(x, np.float32))
    if code in ("bf16", "f32"):
        return t.to(DTYPES[code]), None
    top = torch.full(t.shape[:-1] + (1,), TOP[code])
    a = t.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)
    y = t * (top / a)
    y = y.round().clamp(-127, 127) if code == "i8" else y.clamp(-448, 448)
    return y.to(DTYPES[code]), (a / top)[..., 0]


def values(t):
    """float64 numpy values of a CPU or GPU tensor of any type."""
    return t.detach().cpu().to(torch.float32).to(torch.float64).numpy()


def cuda(a):
    return torch.as_tensor(np.ascontiguousarray(a)).cuda()


def random_tree(g, n, max_depth=16):
    """Parents, depths and ancestor words of a random tree of n nodes."""
    parent, depth, anc = np.full(n, -1), np.ones(n, np.int32), np.zeros(n, np.uint64)
    for i in range(n):
        p = int(g.integers(-1, i)) if i else -1
        while p >= 0 and depth[p] >= max_depth:
            p = int(parent[p])
        parent[i] = p
        depth[i] = 1 if p < 0 else depth[p] + 1
        anc[i] = np.uint64(1 << i) | (anc[p] if p >= 0 else np.uint64(0))
    return parent, depth, anc
