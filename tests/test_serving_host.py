"""The paged-cache, paged-attention and logits entry points refuse bad arguments before touching a
device (no GPU needed), in the library and in the Python surface."""
import ctypes

import pytest
import torch

import draft_tree_construction_markov_b200 as dt
import draft_tree_construction_markov_b200._lib as L

P = ctypes.c_void_p(0x1000)      # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1008)    # not on 16 bytes
EINVAL, EUNSUPPORTED, EWORKSPACE = L.DT_EINVAL, L.DT_EUNSUPPORTED, L.DT_EWORKSPACE


def _cache(**kw):
    f = dict(k=P, v=P, ks=P, vs=P, n_pages=4, page=16, Hkv=2, d=64, dt=L.DT_E4M3)
    f.update(kw)
    return ctypes.byref(L.KvCacheStruct(f["k"], f["v"], f["ks"], f["vs"], f["n_pages"], f["page"],
                                        f["Hkv"], f["d"], f["dt"]))


CACHE_FAULTS = [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(ks=None), EINVAL), (dict(vs=None), EINVAL),
    (dict(dt=9), EINVAL), (dict(n_pages=0), EINVAL), (dict(page=0), EINVAL), (dict(Hkv=0), EINVAL),
    (dict(k=ODD), EINVAL), (dict(page=24), EUNSUPPORTED), (dict(page=4), EUNSUPPORTED),
    (dict(page=512), EUNSUPPORTED), (dict(d=96), EUNSUPPORTED), (dict(Hkv=1025), EUNSUPPORTED),
    (dict(n_pages=1 << 30), EUNSUPPORTED),
]


def _write(cache=None, **kw):
    a = dict(k=P, v=P, ld_k=128, ld_v=128, dt=L.DT_BF16, start=P, pos=P, table=P, max_pages=4, batch=2,
             rows=10, ws=P, bytes=256)
    a.update(kw)
    return L.lib.dt_kv_write(a["k"], a["v"], a["ld_k"], a["ld_v"], a["dt"], a["start"], a["pos"], a["table"],
                             a["max_pages"], a["batch"], a["rows"], cache or _cache(), a["ws"], a["bytes"],
                             None)


def _commit(cache=None, **kw):
    a = dict(k=P, v=P, dt=L.DT_BF16, acc=P, n_acc=P, Bk=4, Nmax=8, pos=P, table=P, max_pages=4, batch=2,
             ws=P, bytes=256)
    a.update(kw)
    return L.lib.dt_kv_commit(a["k"], a["v"], a["dt"], a["acc"], a["n_acc"], a["Bk"], a["Nmax"], a["pos"],
                              a["table"], a["max_pages"], a["batch"], cache or _cache(), a["ws"], a["bytes"],
                              None)


def _read(cache=None, **kw):
    a = dict(table=P, max_pages=4, start=P, pos=P, batch=2, rows=10, dt=L.DT_BF16, k=P, v=P, ws=P, bytes=256)
    a.update(kw)
    return L.lib.dt_kv_read(cache or _cache(), a["table"], a["max_pages"], a["start"], a["pos"], a["batch"],
                            a["rows"], a["dt"], a["k"], a["v"], a["ws"], a["bytes"], None)


def _attn(cache=None, **kw):
    a = dict(q=P, ld=256, start=P, table=P, max_pages=4, kv=P, batch=2, rows=10, max_rows=5, Hq=4, scale=0.1,
             window=0, sink=0, dt=L.DT_BF16, out=P, ws=P, bytes=1 << 40)
    a.update(kw)
    return L.lib.dt_paged_attn(a["q"], a["ld"], a["start"], cache or _cache(), a["table"], a["max_pages"],
                               a["kv"], a["batch"], a["rows"], a["max_rows"], a["Hq"], a["scale"], a["window"],
                               a["sink"], a["dt"], a["out"], a["ws"], a["bytes"], None)


def _tree(cache=None, **kw):
    a = dict(q=P, table=P, max_pages=4, plen=P, k=P, v=P, anc=P, depths=P, n=P, batch=2, Nmax=8, Hq=4,
             scale=0.1, window=0, sink=0, dt=L.DT_BF16, out=P, ws=P, bytes=1 << 40)
    a.update(kw)
    return L.lib.dt_tree_verify_attn_paged(
        a["q"], cache or _cache(), a["table"], a["max_pages"], a["plen"], a["k"], a["v"], a["anc"], a["depths"],
        a["n"], a["batch"], a["Nmax"], a["Hq"], a["scale"], a["window"], a["sink"], a["dt"], a["out"], a["ws"],
        a["bytes"], None)


@pytest.mark.parametrize("call", [_write, _commit, _read, _attn, _tree])
@pytest.mark.parametrize("fault,code", CACHE_FAULTS)
def test_a_bad_cache_is_refused_by_every_call(call, fault, code):
    assert call(_cache(**fault)) == code


@pytest.mark.parametrize("call", [_write, _commit, _read, _attn, _tree])
@pytest.mark.parametrize("fault,code", [
    (dict(table=None), EINVAL), (dict(max_pages=0), EINVAL), (dict(batch=0), EINVAL),
    (dict(batch=1025), EUNSUPPORTED), (dict(max_pages=1 << 26), EUNSUPPORTED), (dict(dt=7), EINVAL),
    (dict(dt=L.DT_I8), EINVAL), (dict(ws=None), EWORKSPACE), (dict(bytes=8), EWORKSPACE)])
def test_shared_arguments(call, fault, code):
    assert call(**fault) == code


@pytest.mark.parametrize("call,fault,code", [
    (_write, dict(k=None), EINVAL), (_write, dict(start=None), EINVAL), (_write, dict(pos=None), EINVAL),
    (_write, dict(rows=-1), EINVAL), (_write, dict(ld_k=127), EINVAL), (_write, dict(ld_v=0), EINVAL),
    (_write, dict(k=ctypes.c_void_p(0x1001)), EINVAL),
    (_commit, dict(acc=None), EINVAL), (_commit, dict(n_acc=None), EINVAL), (_commit, dict(Bk=0), EINVAL),
    (_commit, dict(Bk=65), EUNSUPPORTED), (_commit, dict(Nmax=65), EUNSUPPORTED),
    (_read, dict(k=ODD), EINVAL), (_read, dict(start=None), EINVAL), (_read, dict(rows=-1), EINVAL),
    (_attn, dict(q=None), EINVAL), (_attn, dict(out=None), EINVAL), (_attn, dict(q=ODD), EINVAL),
    (_attn, dict(ld=255), EINVAL), (_attn, dict(ld=260), EINVAL), (_attn, dict(Hq=5), EINVAL),
    (_attn, dict(scale=0.0), EINVAL), (_attn, dict(scale=float("nan")), EINVAL), (_attn, dict(window=-1), EINVAL),
    (_attn, dict(sink=-1), EINVAL), (_attn, dict(max_rows=0), EINVAL), (_attn, dict(rows=1 << 29), EUNSUPPORTED),
    (_attn, dict(kv=None), EINVAL),
    (_tree, dict(Nmax=0), EINVAL), (_tree, dict(Nmax=65), EUNSUPPORTED), (_tree, dict(anc=None), EINVAL),
    (_tree, dict(window=9, depths=None), EINVAL), (_tree, dict(window=8), EUNSUPPORTED),
    (_tree, dict(k=ODD), EINVAL), (_tree, dict(n=None), EINVAL), (_tree, dict(plen=None), EINVAL)])
def test_each_call_s_own_arguments(call, fault, code):
    assert call(**fault) == code


def test_a_bf16_query_has_no_fp32_cache():
    assert _attn(_cache(dt=L.DT_F32)) == EUNSUPPORTED
    assert _tree(_cache(dt=L.DT_F32)) == EUNSUPPORTED


def _logits(**kw):
    a = dict(x=P, dt=1, tokens=P, anc=P, n=P, batch=2, Nmax=8, V=100, hist=P, hstart=P, npr=None, nh=5, rep=None,
             pres=None, freq=None, bs=None, bt=None, bv=None, nb=0, mask=None, mrow=None, nm=0, out=P, ws=P,
             bytes=256)
    a.update(kw)
    return L.lib.dt_logits_process(*list(a.values()), None)


@pytest.mark.parametrize("fault,code", [
    (dict(x=None), EINVAL), (dict(out=None), EINVAL), (dict(dt=2), EINVAL), (dict(batch=0), EINVAL),
    (dict(Nmax=-1), EINVAL), (dict(V=0), EINVAL), (dict(tokens=None), EINVAL), (dict(anc=None), EINVAL),
    (dict(n=None), EINVAL), (dict(Nmax=0), EINVAL), (dict(hstart=None), EINVAL), (dict(hist=None), EINVAL),
    (dict(hist=None, hstart=None, npr=P), EINVAL), (dict(bs=P), EINVAL), (dict(bt=P, bv=P), EINVAL),
    (dict(mrow=P), EINVAL), (dict(nh=-1), EINVAL), (dict(x=ODD, out=ODD), EINVAL),
    (dict(out=ctypes.c_void_p(0x1010)), EINVAL),     # overlaps the input without being it
    (dict(Nmax=65), EUNSUPPORTED), (dict(batch=1025), EUNSUPPORTED), (dict(V=1 << 24), EUNSUPPORTED),
    (dict(ws=None), EWORKSPACE), (dict(bytes=100), EWORKSPACE)])
def test_logits_arguments(fault, code):
    assert _logits(**fault) == code


def test_workspace_queries():
    assert dt.kv_workspace_bytes() >= 256 and dt.logits_workspace_bytes() >= 256
    a = dt.paged_attn_workspace_bytes(4, 100, 32, 8, 128)
    assert 256 <= a <= dt.paged_attn_workspace_bytes(4, 10000, 32, 8, 128)
    assert dt.paged_attn_workspace_bytes(0, 1, 2, 1, 64) == 0
    assert dt.paged_attn_workspace_bytes(1, 1, 3, 2, 64) == 0
    assert dt.verify_paged_workspace_bytes(1, 64, 32, 8, 128) >= 256
    assert dt.verify_paged_workspace_bytes(1, 0, 32, 8, 128) == 0


def _cpu_cache(dtype=torch.int8):
    return dt.KVCache.empty(4, 16, 2, 64, dtype, device="cpu")


def test_the_python_cache_checks_its_tensors():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    s = torch.zeros(4, 2, 16)
    dt.KVCache(k, k, s, s)
    for bad in ((k, k), (k, k, s, None), (k.float(), k.float(), s, s), (k, k[:3], s, s), (k, k, s[:3], s),
                (k.transpose(1, 2), k.transpose(1, 2), s, s), (k[0], k[0], s, s)):
        with pytest.raises(ValueError):
            dt.KVCache(*bad)
    with pytest.raises(TypeError):
        dt.KVCache(k.to(torch.float16), k.to(torch.float16))
    with pytest.raises(TypeError):
        dt.KVCache(k, k, s.double(), s.double())


def test_the_python_calls_check_their_tensors():
    c = _cpu_cache()
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    x = torch.zeros(10, 2, 64)
    q = torch.zeros(10, 4, 64, dtype=torch.bfloat16)
    for call in (
        lambda: dt.kv_write(x, x, i(2), i(2), c, i(2, 4), ws),                 # batch + 1 starts
        lambda: dt.kv_write(x, x, i(3), i(1), c, i(2, 4), ws),
        lambda: dt.kv_write(x[:, :1], x[:, :1], i(3), i(2), c, i(2, 4), ws),   # heads
        lambda: dt.kv_write(x.transpose(0, 1), x, i(3), i(2), c, i(2, 4), ws),
        lambda: dt.kv_write(x, x, i(3), i(2), c, i(8), ws),                    # table is a row
        lambda: dt.kv_read(c, i(2, 4), i(3), i(2), x, x[:9], ws),
        lambda: dt.kv_commit(x, x, i(2, 4), i(2), i(2), c, i(2, 4), ws),
        lambda: dt.paged_attn(q, i(3), c, i(2, 4), i(3), 0.1, q, ws, max_rows=5),
        lambda: dt.paged_attn(q, i(3), c, i(2, 4), i(2), 0.1, q[:9], ws, max_rows=5),
        lambda: dt.paged_attn(q, i(3), c, i(2, 4).T.contiguous().T, i(2), 0.1, q, ws, max_rows=5),
    ):
        with pytest.raises((ValueError, IndexError)):
            call()
    with pytest.raises(TypeError):
        dt.kv_write(x, x, i(3).long(), i(2), c, i(2, 4), ws)
    t = torch.zeros(2, 9, 4, 64, dtype=torch.bfloat16)
    kt = torch.zeros(2, 9, 2, 64, dtype=torch.bfloat16)
    anc = torch.zeros(2, 8, dtype=torch.int64)
    with pytest.raises(ValueError):
        dt.tree_verify_attn_paged(t, c, i(2, 4), i(2), kt, kt, anc[:, :7].contiguous(), i(2), 0.1, t, ws)
    with pytest.raises(TypeError):
        dt.tree_verify_attn_paged(t, c, i(2, 4), i(2), kt.float(), kt, anc, i(2), 0.1, t, ws)
    z = torch.zeros(2, 1, 50)
    with pytest.raises(ValueError):
        dt.logits_process(z, z[:1], ws)
    with pytest.raises(ValueError):
        dt.logits_process(z, z, ws, history=i(5), history_start=i(2))
    with pytest.raises(ValueError):
        dt.logits_process(z, z, ws, mask=i(2, 3))
    with pytest.raises(TypeError):
        dt.logits_process(z, z, ws, repetition=torch.ones(2).double())
