"""B200 (sm_100a) draft-tree round: tree_build, tree_verify_attn, tree_accept.

Thin Python surface over libdtree.so (see include/dtree.h for the exact
semantics, layouts and error behaviour of every call).  Tensors must be CUDA
tensors; the library allocates nothing, so each call takes a workspace tensor
(``workspace(...)`` allocates one of the right size).
"""
import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import DtreeError, check, dtype_code, ptr, stream_ptr

__all__ = ["Tree", "tree_build", "tree_verify_attn", "tree_accept", "markov_logits",
           "read_status", "build_workspace_bytes", "verify_workspace_bytes",
           "accept_workspace_bytes", "workspace", "DtreeError", "num_sms", "tree_load_budget",
           "load_budget_workspace_bytes", "calib_workspace_bytes", "calib_log", "calib_fit",
           "tree_accept_noalloc",
           "shard_range", "shard_cfg", "sharded_workspace_bytes", "sharded_partials_bytes",
           "sharded_build_begin", "sharded_build_gemm", "sharded_build_frontier",
           "tree_build_sharded", "set_build_path", "set_build_wait_test",
           "KVCache", "kv_workspace_bytes", "kv_write", "kv_commit", "kv_read",
           "paged_attn_workspace_bytes", "paged_attn", "verify_paged_workspace_bytes",
           "tree_verify_attn_paged", "logits_workspace_bytes", "logits_process"]


def num_sms() -> int:
    return int(_lib.lib.dt_num_sms())


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Device scratch for one call site; its 256-byte header (the status word
    that read_status returns) starts cleared."""
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


@dataclass
class Tree:
    """Device arrays of a batch of draft trees (dt_tree in the C header)."""
    tokens: torch.Tensor      # [batch, Nmax] int32
    parents: torch.Tensor     # [batch, Nmax] int32
    depths: torch.Tensor      # [batch, Nmax] int32
    ranks: torch.Tensor       # [batch, Nmax] int32
    keys: torch.Tensor        # [batch, Nmax] float32
    anc: torch.Tensor         # [batch, Nmax] int64 (uint64 bit patterns)
    n_nodes: torch.Tensor     # [batch] int32
    draft_q: Optional[torch.Tensor] = None   # [batch, Nmax+1, V] float32 (T > 0)

    @staticmethod
    def empty(batch, Nmax, V=None, stochastic=False, device="cuda"):
        i = dict(dtype=torch.int32, device=device)
        return Tree(
            tokens=torch.zeros(batch, Nmax, **i), parents=torch.zeros(batch, Nmax, **i),
            depths=torch.zeros(batch, Nmax, **i), ranks=torch.zeros(batch, Nmax, **i),
            keys=torch.zeros(batch, Nmax, dtype=torch.float32, device=device),
            anc=torch.zeros(batch, Nmax, dtype=torch.int64, device=device),
            n_nodes=torch.zeros(batch, **i),
            draft_q=(torch.zeros(batch, Nmax + 1, V, dtype=torch.float32, device=device)
                     if stochastic else None))

    def c_struct(self):
        return _lib.DtTree(*(ctypes.c_void_p(t.data_ptr()) if t is not None else None for t in
                             (self.tokens, self.parents, self.depths, self.ranks, self.keys,
                              self.anc, self.n_nodes, self.draft_q)))


def build_workspace_bytes(batch, Bk, V, r, k, Nmax) -> int:
    return int(_lib.lib.dt_tree_build_workspace_bytes(batch, Bk, V, r, k, Nmax))


def verify_workspace_bytes(batch, Nmax, Hq, Hkv, d, max_prefix) -> int:
    return int(_lib.lib.dt_tree_verify_attn_workspace_bytes(batch, Nmax, Hq, Hkv, d, max_prefix))


def accept_workspace_bytes(batch, Nmax, V) -> int:
    return int(_lib.lib.dt_tree_accept_workspace_bytes(batch, Nmax, V))


def tree_build(block_logits, markov_a, markov_b, root_token, n_budget, lam, *, k, Nmax, temp,
               out: Tree, ws, calib=None, k_req=None, philox_seed=0, philox_offset=0,
               stream=None, variant="pctree"):
    """dt_tree_build (variant "pctree") or dt_tree_build_ex with a baseline
    variant ("chain", "marginal", "shared_markov").  block_logits
    [batch,Bk,V] fp32|bf16; markov_a/markov_b [V,r] bf16."""
    batch, Bk, V = block_logits.shape
    r = markov_a.shape[1]
    st = out.c_struct()
    args = (ptr(block_logits), dtype_code(block_logits), ptr(markov_a), ptr(markov_b), r,
            ptr(calib), ptr(root_token), ptr(n_budget), ptr(k_req), ptr(lam), batch, Bk, V, k,
            Nmax, float(temp), philox_seed, philox_offset)
    tail = (ctypes.byref(st), ptr(ws), ws.numel(), stream_ptr(stream))
    if variant == "pctree":
        check(_lib.lib.dt_tree_build(*args, *tail), "dt_tree_build")
    else:
        check(_lib.lib.dt_tree_build_ex(*args, _lib.TREE_VARIANTS[variant], *tail),
              "dt_tree_build_ex")
    return out


def markov_logits(block_logits, markov_a, markov_b, req, depth, token, out, ws, stream=None):
    """dt_markov_logits: z rows [n_rows, V] fp32 for (request, depth, token) triples."""
    batch, Bk, V = block_logits.shape
    check(_lib.lib.dt_markov_logits(
        ptr(block_logits), dtype_code(block_logits), ptr(markov_a), ptr(markov_b),
        markov_a.shape[1], batch, Bk, V, ptr(req), ptr(depth), ptr(token), req.numel(), ptr(out),
        ptr(ws), ws.numel(), stream_ptr(stream)), "dt_markov_logits")
    return out


def tree_verify_attn(q, k_prefix, v_prefix, prefix_start, prefix_len, max_prefix, k_tree, v_tree,
                     anc, n_nodes, scale, out, ws, stream=None):
    """dt_tree_verify_attn.  q/out [batch,Nmax+1,Hq,d]; k/v_prefix [rows,Hkv,d]."""
    batch, n1, Hq, d = q.shape
    Hkv = k_prefix.shape[1]
    check(_lib.lib.dt_tree_verify_attn(
        ptr(q), ptr(k_prefix), ptr(v_prefix), ptr(prefix_start), ptr(prefix_len), int(max_prefix),
        ptr(k_tree), ptr(v_tree), ptr(anc), ptr(n_nodes), batch, n1 - 1, Hq, Hkv, d, float(scale),
        dtype_code(q), ptr(out), ptr(ws), ws.numel(), stream_ptr(stream)), "dt_tree_verify_attn")
    return out


def tree_accept(target_logits, tree: Tree, Bk, temp, acc_nodes, n_acc, bonus, ws,
                philox_seed=0, philox_offset=0, stream=None):
    """dt_tree_accept.  target_logits [batch,Nmax+1,V] fp32|bf16."""
    batch, n1, V = target_logits.shape
    st = tree.c_struct()
    check(_lib.lib.dt_tree_accept(
        ptr(target_logits), dtype_code(target_logits), ctypes.byref(st), batch, Bk, V, n1 - 1,
        float(temp), philox_seed, philox_offset, ptr(acc_nodes), ptr(n_acc), ptr(bonus), ptr(ws),
        ws.numel(), stream_ptr(stream)), "dt_tree_accept")
    return acc_nodes, n_acc, bonus


def tree_accept_noalloc(target_logits, tree: Tree, Bk, temp, acc_nodes, n_acc, bonus,
                        philox_seed=0, philox_offset=0, stream=None):
    """dt_tree_accept_noalloc: dt_tree_accept with the library's fixed scratch
    (no workspace; batch 1 at V = 151936 fits, larger sizes raise
    DT_EUNSUPPORTED)."""
    batch, n1, V = target_logits.shape
    st = tree.c_struct()
    check(_lib.lib.dt_tree_accept_noalloc(
        ptr(target_logits), dtype_code(target_logits), ctypes.byref(st), batch, Bk, V, n1 - 1,
        float(temp), philox_seed, philox_offset, ptr(acc_nodes), ptr(n_acc), ptr(bonus),
        stream_ptr(stream)), "dt_tree_accept_noalloc")
    return acc_nodes, n_acc, bonus


def treeflash_workspace_bytes(batch, gamma, D, Dff, V, M, budget) -> int:
    return int(_lib.lib.dt_treeflash_workspace_bytes(batch, gamma, D, Dff, V, M, budget))


def treeflash_build(h, embed, w_norm_h, w_norm_e, w_gate, w_up, w_down, w_lm, root, *, M,
                    budget, out: Tree, ws, stream=None):
    """dt_treeflash_build.  h [batch,gamma,D] bf16; embed/w_lm [V,D] bf16; w_gate/w_up
    [Dff,2D] bf16; w_down [D,Dff] bf16; w_norm_h/w_norm_e [D] fp32; root [batch] int32."""
    batch, gamma, D = h.shape
    V = w_lm.shape[0]
    Dff = w_gate.shape[0]
    st = out.c_struct()
    check(_lib.lib.dt_treeflash_build(
        ptr(h), ptr(embed), ptr(w_norm_h), ptr(w_norm_e), ptr(w_gate), ptr(w_up), ptr(w_down),
        ptr(w_lm), ptr(root), batch, gamma, D, Dff, V, M, budget, ctypes.byref(st), ptr(ws),
        ws.numel(), stream_ptr(stream)), "dt_treeflash_build")
    return out


def tree_load_budget(tree: Tree, capacity, ws, *, prefix_len=None, prefix_unit=0, n_keep=None,
                     stream=None):
    """dt_tree_load_budget: cut the batch's trees (in place) to a round's
    verification capacity by survival; returns ``tree``."""
    batch, Nmax = tree.keys.shape
    st = tree.c_struct()
    check(_lib.lib.dt_tree_load_budget(
        ctypes.byref(st), batch, Nmax, ptr(prefix_len), int(capacity), int(prefix_unit),
        ptr(n_keep), ptr(ws), ws.numel(), stream_ptr(stream)), "dt_tree_load_budget")
    return tree


def load_budget_workspace_bytes() -> int:
    return int(_lib.lib.dt_tree_load_budget_workspace_bytes())


def calib_workspace_bytes(Bk=1, n_alpha=1, n_beta=1) -> int:
    return int(_lib.lib.dt_calib_workspace_bytes(Bk, n_alpha, n_beta))


def calib_log(tree: Tree, acc_nodes, n_acc, Bk, depth, ell, y, ws, stream=None):
    """dt_calib_log: (depth, l, y) [batch, Nmax] of every child of a reached node."""
    batch, Nmax = tree.keys.shape
    st = tree.c_struct()
    check(_lib.lib.dt_calib_log(
        ctypes.byref(st), ptr(acc_nodes), ptr(n_acc), batch, Bk, Nmax, ptr(depth), ptr(ell), ptr(y),
        ptr(ws), ws.numel(), stream_ptr(stream)), "dt_calib_log")
    return depth, ell, y


def calib_fit(depth, ell, y, Bk, grid, calib, ws, loglik=None, min_samples=1, stream=None):
    """dt_calib_fit over the flattened samples; grid = (alpha0, dalpha, n_alpha,
    beta0, dbeta, n_beta); writes calib [Bk, 2] fp32 (and loglik [Bk] fp64)."""
    a0, da, na, b0, db, nb = grid
    check(_lib.lib.dt_calib_fit(
        ptr(depth), ptr(ell), ptr(y), depth.numel(), Bk, float(a0), float(da), int(na), float(b0),
        float(db), int(nb), int(min_samples), ptr(calib), ptr(loglik), ptr(ws), ws.numel(),
        stream_ptr(stream)), "dt_calib_fit")
    return calib


# ------------------------------------------------ vocabulary-sharded build --
def shard_range(V, world, rank):
    """(v_base, v_len): the Markov-factor rows Bm[v_base : v_base + v_len] rank holds."""
    a, b = ctypes.c_int(0), ctypes.c_int(0)
    _lib.lib.dt_shard_range(V, world, rank, ctypes.byref(a), ctypes.byref(b))
    return a.value, b.value


def shard_cfg(batch, Bk, V, r, k, Nmax, world, ncta=None):
    ncta = int(_lib.lib.dt_shard_ncta(V, world)) if ncta is None else ncta
    return _lib.ShardCfg(batch, Bk, V, r, k, Nmax, world, ncta)


def sharded_workspace_bytes(cfg) -> int:
    return int(_lib.lib.dt_sharded_workspace_bytes(ctypes.byref(cfg)))


def sharded_partials_bytes(cfg) -> int:
    return int(_lib.lib.dt_sharded_partials_bytes(ctypes.byref(cfg)))


def sharded_build_begin(cfg, root_token, n_budget, lam, out: Tree, ws, k_req=None, stream=None):
    st = out.c_struct()
    check(_lib.lib.dt_sharded_build_begin(
        ctypes.byref(cfg), ptr(root_token), ptr(n_budget), ptr(k_req), ptr(lam), ctypes.byref(st),
        ptr(ws), ws.numel(), stream_ptr(stream)), "dt_sharded_build_begin")


def sharded_build_gemm(cfg, wave, rank, block_logits, markov_a, markov_b_shard, ws, partials,
                       stream=None):
    check(_lib.lib.dt_sharded_build_gemm(
        ctypes.byref(cfg), wave, rank, ptr(block_logits), dtype_code(block_logits), ptr(markov_a),
        ptr(markov_b_shard), ptr(ws), ws.numel(), ptr(partials), stream_ptr(stream)),
        "dt_sharded_build_gemm")


def sharded_build_frontier(cfg, wave, gathered, n_budget, lam, out: Tree, ws, calib=None,
                           k_req=None, stream=None):
    st = out.c_struct()
    check(_lib.lib.dt_sharded_build_frontier(
        ctypes.byref(cfg), wave, ptr(gathered), ptr(calib), ptr(n_budget), ptr(k_req), ptr(lam),
        ctypes.byref(st), ptr(ws), ws.numel(), stream_ptr(stream)), "dt_sharded_build_frontier")


def tree_build_sharded(cfg, rank, block_logits, markov_a, markov_b_shard, root_token, n_budget,
                       lam, out: Tree, ws, partials, gathered, all_gather, calib=None, k_req=None,
                       stream=None):
    """The sharded build's wave loop on one rank.  ``partials`` holds this
    rank's block (sharded_partials_bytes), ``gathered`` world blocks;
    ``all_gather(gathered, partials)`` must fill ``gathered`` with every
    rank's block in rank order (torch.distributed.all_gather_into_tensor over
    the ranks sharing the vocabulary)."""
    sharded_build_begin(cfg, root_token, n_budget, lam, out, ws, k_req=k_req, stream=stream)
    for wave in range(cfg.Bk):
        sharded_build_gemm(cfg, wave, rank, block_logits, markov_a, markov_b_shard, ws, partials,
                           stream=stream)
        all_gather(gathered, partials)
        sharded_build_frontier(cfg, wave, gathered, n_budget, lam, out, ws, calib=calib,
                               k_req=k_req, stream=stream)
    return out


# -------------------------------------------------------- paged KV cache --
_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32
_FLOATS = {torch.float32: _lib.DT_F32, torch.bfloat16: _lib.DT_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _arg(where, name, t, dev, dtype, *shape):
    """Address of a contiguous tensor of this device, type and shape.  (A serving step makes
    several of these calls back to back: the checks are few and cheap.)"""
    if t.dtype is not dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} must have shape {shape}, not {tuple(t.shape)}")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous and on the device of the others")
    return t.data_ptr()


def _opt(where, name, t, dev, dtype, *shape):
    return None if t is None else _arg(where, name, t, dev, dtype, *shape)


def _float_code(where, name, t):
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"{where}: {name} must be float32 or bfloat16, not {t.dtype}")
    return code


def _workspace(where, ws, dev):
    if ws.get_device() != dev or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"{where}: ws must be a contiguous uint8 tensor on the others' device")
    return ws.data_ptr(), ws.numel()


def _run(fn, where, dev, stream, *args):
    """Call ``fn`` with device ``dev`` current and the stream as its last argument."""
    if dev < 0:
        raise ValueError(f"{where}: the tensors must be on a CUDA device")
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _run(fn, where, dev, stream, *args)
    code = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if code:
        check(code, where)


def _row_stride(where, name, t, dev, heads, d):
    """Elements between the rows of a [rows, heads, d] tensor whose rows are whole."""
    if t.dim() != 3 or t.shape[1:] != (heads, d):
        raise ValueError(f"{where}: {name} must have shape (rows, {heads}, {d})")
    ld, head, one = t.stride()
    if one != 1 or (heads > 1 and head != d):
        raise ValueError(f"{where}: the heads of a row of {name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{where}: {name} must be on the device of the others")
    return ld if t.shape[0] > 1 else max(ld, heads * d)


class KVCache:
    """A paged pool of keys and values (dt_kv_cache in the C header).

    ``k``, ``v``: [n_pages, Hkv, page_size, d], bfloat16, float32, float8_e4m3fn or int8;
    ``k_scale``, ``v_scale``: [n_pages, Hkv, page_size] float32 for the 8-bit types, else None.
    The tensors are the caller's to fill, but not to exchange: the attributes cannot be set (a larger
    pool is another KVCache), and a call on tensors whose storage has moved raises."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        code = _lib.cache_dtype_code(k)
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("KVCache: k and v must be [n_pages, Hkv, page_size, d] of one type")
        dev = k.get_device()
        scaled = code in (_lib.DT_E4M3, _lib.DT_I8)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if scaled != (t is not None):
                raise ValueError(f"KVCache: {name} goes with the 8-bit types, and only with them")
        at = [_arg("KVCache", name, t, dev, k.dtype, *k.shape) for name, t in (("k", k), ("v", v))]
        at += [_opt("KVCache", name, t, dev, _F32, *k.shape[:3])
               for name, t in (("k_scale", k_scale), ("v_scale", v_scale))]
        n_pages, Hkv, page_size, d = k.shape
        c = _lib.KvCacheStruct(*at, n_pages, page_size, Hkv, d, code)
        self.__dict__.update(
            k=k, v=v, k_scale=k_scale, v_scale=v_scale, n_pages=n_pages, Hkv=Hkv, page_size=page_size, d=d,
            device=dev, _c=c, _ref=ctypes.byref(c), _at=(k, v, k_scale, v_scale, *at))

    def __setattr__(self, name, value):
        raise AttributeError(f"KVCache: {name} cannot be set; make a new KVCache")

    @staticmethod
    def empty(n_pages, page_size, Hkv, d, dtype=torch.bfloat16, device="cuda"):
        shape = (n_pages, Hkv, page_size, d)
        new = lambda: torch.zeros(shape, dtype=dtype, device=device)
        scale = lambda: (torch.zeros(shape[:3], dtype=torch.float32, device=device)
                         if dtype in (torch.float8_e4m3fn, torch.int8) else None)
        return KVCache(new(), new(), scale(), scale())


def _table(where, cache, t):
    """Address and shape of a page table; looks whether the cache is still where it was."""
    k, v, ks, vs, at_k, at_v, at_ks, at_vs = cache._at
    if (k.data_ptr() != at_k or v.data_ptr() != at_v
            or ks is not None and (ks.data_ptr() != at_ks or vs.data_ptr() != at_vs)):
        raise ValueError(f"{where}: the cache's tensors have moved; make a new KVCache")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{where}: page_table must be [batch, max_pages]")
    if t.dtype is not _I32 or t.get_device() != cache.device or not t.is_contiguous():
        _arg(where, "page_table", t, cache.device, _I32, *shape)  # says what is wrong
    return t.data_ptr(), *shape


def kv_workspace_bytes() -> int:
    return int(_lib.lib.dt_kv_workspace_bytes())


def kv_write(k, v, row_start, pos, cache, page_table, ws, stream=None):
    """dt_kv_write: rows row_start[b] + i of k/v [rows, Hkv, d] (fp32 or bf16, any row stride) to
    positions pos[b] + i of request b; returns ``cache``."""
    where, dev = "kv_write", cache.device
    table, batch, pages = _table(where, cache, page_table)
    starts = _arg(where, "row_start", row_start, dev, _I32, batch + 1)
    first = _arg(where, "pos", pos, dev, _I32, batch)
    if v.shape != k.shape or v.dtype is not k.dtype:
        raise ValueError("kv_write: k and v must have one shape and type")
    ld_k = _row_stride(where, "k", k, dev, cache.Hkv, cache.d)
    ld_v = _row_stride(where, "v", v, dev, cache.Hkv, cache.d)
    rows = k.shape[0]
    if rows:
        _run(_lib.lib.dt_kv_write, where, dev, stream, k.data_ptr(), v.data_ptr(), ld_k, ld_v,
             _float_code(where, "k", k), starts, first, table, pages, batch, rows, cache._ref,
             *_workspace(where, ws, dev))
    return cache


def kv_commit(k_tree, v_tree, acc_nodes, n_acc, pos, cache, page_table, ws, stream=None):
    """dt_kv_commit: the root's and the accepted nodes' rows of k/v_tree [batch, Nmax+1, Hkv, d]
    to positions pos[b], pos[b] + 1, ...; returns ``cache``."""
    where, dev = "kv_commit", cache.device
    table, batch, pages = _table(where, cache, page_table)
    n1, Bk, dtype = k_tree.shape[1], acc_nodes.shape[1], k_tree.dtype
    shape = batch, n1, cache.Hkv, cache.d
    _run(_lib.lib.dt_kv_commit, where, dev, stream, _arg(where, "k_tree", k_tree, dev, dtype, *shape),
         _arg(where, "v_tree", v_tree, dev, dtype, *shape), _float_code(where, "k_tree", k_tree),
         _arg(where, "acc_nodes", acc_nodes, dev, _I32, batch, Bk),
         _arg(where, "n_acc", n_acc, dev, _I32, batch), Bk, n1 - 1,
         _arg(where, "pos", pos, dev, _I32, batch), table, pages, batch, cache._ref,
         *_workspace(where, ws, dev))
    return cache


def kv_read(cache, page_table, row_start, pos, k_out, v_out, ws, stream=None):
    """dt_kv_read: positions pos[b] + i into rows row_start[b] + i of k/v_out [rows, Hkv, d], the
    packed prefix that tree_verify_attn takes (prefix_start = row_start)."""
    where, dev, dtype = "kv_read", cache.device, k_out.dtype
    table, batch, pages = _table(where, cache, page_table)
    rows = k_out.shape[0]
    shape = rows, cache.Hkv, cache.d
    starts = _arg(where, "row_start", row_start, dev, _I32, batch + 1)
    first = _arg(where, "pos", pos, dev, _I32, batch)
    to_k = _arg(where, "k_out", k_out, dev, dtype, *shape)
    to_v = _arg(where, "v_out", v_out, dev, dtype, *shape)
    if rows:
        _run(_lib.lib.dt_kv_read, where, dev, stream, cache._ref, table, pages, starts, first, batch,
             rows, _float_code(where, "k_out", k_out), to_k, to_v, *_workspace(where, ws, dev))
    return k_out, v_out


def paged_attn_workspace_bytes(batch, total_rows, Hq, Hkv, d) -> int:
    return int(_lib.lib.dt_paged_attn_workspace_bytes(batch, total_rows, Hq, Hkv, d))


def paged_attn(q, row_start, cache, page_table, kv_len, scale, out, ws, *, max_rows, window=0,
               n_sink=0, stream=None):
    """dt_paged_attn: causal attention of the chunk rows q [rows, Hq, d] (row_start[b] ..
    row_start[b+1] are request b's last tokens) over kv_len[b] cached positions.  window 0 = none;
    with one, the first n_sink positions stay visible.  No request has more than max_rows rows."""
    where, dev = "paged_attn", cache.device
    table, batch, pages = _table(where, cache, page_table)
    starts = _arg(where, "row_start", row_start, dev, _I32, batch + 1)
    lens = _arg(where, "kv_len", kv_len, dev, _I32, batch)
    if q.dim() != 3:
        raise ValueError("paged_attn: q must be [rows, Hq, d]")
    total, Hq, _ = q.shape
    ld = _row_stride(where, "q", q, dev, Hq, cache.d)
    to = _arg(where, "out", out, dev, q.dtype, total, Hq, cache.d)
    if total:
        _run(_lib.lib.dt_paged_attn, where, dev, stream, q.data_ptr(), ld, starts, cache._ref, table,
             pages, lens, batch, total, max_rows, Hq, scale, window, n_sink,
             _float_code(where, "q", q), to, *_workspace(where, ws, dev))
    return out


def verify_paged_workspace_bytes(batch, Nmax, Hq, Hkv, d) -> int:
    return int(_lib.lib.dt_tree_verify_attn_paged_workspace_bytes(batch, Nmax, Hq, Hkv, d))


def tree_verify_attn_paged(q, cache, page_table, prefix_len, k_tree, v_tree, anc, n_nodes, scale,
                           out, ws, *, depths=None, window=0, n_sink=0, stream=None):
    """dt_tree_verify_attn_paged: tree_verify_attn over prefix_len[b] cached positions.  q/out
    [batch, Nmax+1, Hq, d]; k/v_tree [batch, Nmax+1, Hkv, d]; depths only with a window."""
    where, dev, dtype = "tree_verify_attn_paged", cache.device, q.dtype
    table, batch, pages = _table(where, cache, page_table)
    _, n1, Hq, d = q.shape
    rows = batch, n1, cache.Hkv, cache.d
    _run(_lib.lib.dt_tree_verify_attn_paged, where, dev, stream,
         _arg(where, "q", q, dev, dtype, batch, n1, Hq, cache.d), cache._ref, table, pages,
         _arg(where, "prefix_len", prefix_len, dev, _I32, batch),
         _arg(where, "k_tree", k_tree, dev, dtype, *rows),
         _arg(where, "v_tree", v_tree, dev, dtype, *rows),
         _arg(where, "anc", anc, dev, _I64, batch, n1 - 1),
         _opt(where, "depths", depths, dev, _I32, batch, n1 - 1),
         _arg(where, "n_nodes", n_nodes, dev, _I32, batch), batch, n1 - 1, Hq, scale, window, n_sink,
         _float_code(where, "q", q), _arg(where, "out", out, dev, dtype, batch, n1, Hq, cache.d),
         *_workspace(where, ws, dev))
    return out


# ----------------------------------------------------- logits processing --
def logits_workspace_bytes() -> int:
    return int(_lib.lib.dt_logits_workspace_bytes())


def logits_process(logits, out, ws, *, tokens=None, anc=None, n_nodes=None, history=None,
                   history_start=None, n_prompt=None, repetition=None, presence=None,
                   frequency=None, bias_start=None, bias_token=None, bias_value=None, mask=None,
                   mask_row=None, stream=None):
    """dt_logits_process: penalties, biases and masks on logits [batch, Nmax+1, V] (a tree's rows,
    with its tokens, anc and n_nodes) or [batch, 1, V] (no tree); ``out`` may be ``logits``.
    mask [rows, ceil(V / 32)] int32 words, one bit per allowed token."""
    where, dev = "logits_process", logits.get_device()
    batch, n1, V = logits.shape
    # An empty list has no address: what points into it stands for it (the library reads no entry of
    # it, but what points), and without that it is no list.
    n_hist = 0 if history is None else history.shape[0]
    n_bias = 0 if bias_token is None else bias_token.shape[0]
    n_mask = 0 if mask is None else mask.shape[0]
    hist_at = _opt(where, "history_start", history_start, dev, _I32, batch + 1)
    hist = (_arg(where, "history", history, dev, _I32, n_hist) if n_hist else
            None if history is None else hist_at)
    if hist is None and history is not None:
        n_prompt = None
    bias_at = _opt(where, "bias_start", bias_start, dev, _I32, batch + 1)
    token = (_arg(where, "bias_token", bias_token, dev, _I32, n_bias) if n_bias else
             None if bias_token is None else bias_at)
    value = (bias_at if bias_token is not None and not n_bias and (bias_value is None or not len(bias_value)) else
             _opt(where, "bias_value", bias_value, dev, _F32, n_bias))
    mask_at = _opt(where, "mask_row", mask_row, dev, _I32, batch, n1)
    words = (_arg(where, "mask", mask, dev, _I32, n_mask, (V + 31) // 32) if n_mask else
             None if mask is None else mask_at)
    _run(_lib.lib.dt_logits_process, where, dev, stream,
         _arg(where, "logits", logits, dev, logits.dtype, batch, n1, V),
         _float_code(where, "logits", logits),
         _opt(where, "tokens", tokens, dev, _I32, batch, n1 - 1),
         _opt(where, "anc", anc, dev, _I64, batch, n1 - 1),
         _opt(where, "n_nodes", n_nodes, dev, _I32, batch), batch, n1 - 1, V,
         hist, hist_at,
         _opt(where, "n_prompt", n_prompt, dev, _I32, batch), n_hist,
         _opt(where, "repetition", repetition, dev, _F32, batch),
         _opt(where, "presence", presence, dev, _F32, batch),
         _opt(where, "frequency", frequency, dev, _F32, batch),
         bias_at, token, value, n_bias, words, mask_at, n_mask,
         _arg(where, "out", out, dev, logits.dtype, batch, n1, V), *_workspace(where, ws, dev))
    return out


def set_build_path(path: str) -> None:
    """How tree_build runs its waves on this host thread: "auto", "waves" or
    "persistent" (dt_set_build_path)."""
    _lib.lib.dt_set_build_path(_lib.BUILD_PATHS[path])


def set_build_wait_test(stall_cta: int, wait_ns: int) -> None:
    """Test hook: the next persistent build on this thread stalls one CTA at its
    first grid barrier and bounds every wait by wait_ns (dt_set_build_wait_test)."""
    _lib.lib.dt_set_build_wait_test(int(stall_cta), int(wait_ns))


def read_status(ws, stream=None) -> int:
    """Synchronise and return (then clear) the device status word of a workspace."""
    v = ctypes.c_int32(0)
    check(_lib.lib.dt_read_status(ptr(ws), stream_ptr(stream), ctypes.byref(v)), "dt_read_status")
    return int(v.value)
