"""Refusals of the 8-bit cache, dense paged attention and block calls, on the CPU: every one is
decided on the host before any launch, and the binding checks its tensors before the library."""
import ctypes

import pytest
import torch

from hash_hierarchical_top_b200 import build, hhr

P = ctypes.c_void_p(256)      # never dereferenced: validation fails first
BAD = ctypes.c_void_p(256 + 8)
F = ctypes.c_float(0.1)
INV, UNS, WS = hhr.HHR_ERR_INVALID_ARG, hhr.HHR_ERR_UNSUPPORTED, hhr.HHR_ERR_WORKSPACE
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    build.build()
    return hhr.lib()


def _d(**kw):
    base = dict(batch=2, n_q_heads=32, n_kv_heads=8, page_size=32, max_pages_per_seq=4096,
                n_phys_pages=8192)
    base.update(kw)
    return hhr.make_dims(**base)


BAD_DIMS = [dict(head_dim=64), dict(n_q_heads=30), dict(page_size=0), dict(page_size=512),
            dict(batch=0), dict(max_pages_per_seq=40000), dict(n_phys_pages=0)]


def append(L, d, **kw):
    a = dict(k_new=P, v_new=P, stride=8 * 128, start=P, n_new=P, max_new=4, pt=P, k=P, v=P, ke=P, ve=P,
             mean=P)
    a.update(kw)
    return L.hhr_append_kv8(ctypes.byref(d), a["k_new"], a["v_new"], a["stride"], a["start"], a["n_new"],
                            a["max_new"], a["pt"], a["k"], a["v"], a["ke"], a["ve"], a["mean"], None)


def read(L, d, **kw):
    a = dict(k=P, v=P, ke=P, ve=P, pt=P, start=P, n=P, max_n=4, ko=P, vo=P)
    a.update(kw)
    return L.hhr_read_kv8(ctypes.byref(d), a["k"], a["v"], a["ke"], a["ve"], a["pt"], a["start"], a["n"],
                          a["max_n"], a["ko"], a["vo"], None)


def paged(L, d, **kw):
    a = dict(q=P, k_new=None, v_new=None, k=P, v=P, ke=None, ve=None, pt=P, seq=P, scale=F, out=P,
             bf16=0, lse=None, ws=P, n=BIG)
    a.update(kw)
    return L.hhr_paged_attn(ctypes.byref(d), a["q"], a["k_new"], a["v_new"], a["k"], a["v"], a["ke"], a["ve"],
                            a["pt"], a["seq"], a["scale"], a["out"], a["bf16"], a["lse"], a["ws"], a["n"],
                            None)


def select(L, d, **kw):
    a = dict(T=4, q=P, seq=P, pos=P, pt=P, mean=P, m=16, opts=None, blocks=P, count=P, ws=P, n=BIG)
    a.update(kw)
    opts = ctypes.byref(a["opts"]) if a["opts"] is not None else None
    return L.hhr_block_select(ctypes.byref(d), a["T"], a["q"], a["seq"], a["pos"], a["pt"], a["mean"],
                              a["m"], opts, a["blocks"], a["count"], a["ws"], a["n"], None)


def block(L, d, **kw):
    a = dict(T=4, q=P, k=P, v=P, ke=None, ve=None, pt=P, seq=P, pos=P, blocks=P, count=P, m=16,
             scale=F, out=P, bf16=0, lse=None, ws=P, n=BIG)
    a.update(kw)
    return L.hhr_block_attn(ctypes.byref(d), a["T"], a["q"], a["k"], a["v"], a["ke"], a["ve"], a["pt"],
                            a["seq"], a["pos"], a["blocks"], a["count"], a["m"], a["scale"], a["out"],
                            a["bf16"], a["lse"], a["ws"], a["n"], None)


@pytest.mark.parametrize("bad", BAD_DIMS)
@pytest.mark.parametrize("call", [append, read, paged, select, block])
def test_bad_dims(L, call, bad):
    assert call(L, _d(**bad)) in (INV, UNS)


def test_bad_dims_have_no_workspace(L):
    for bad in BAD_DIMS + [dict(n_q_heads=72)]:
        d = _d(**bad)
        assert hhr.hhr_paged_attn_workspace_bytes(d) == 0
        assert hhr.hhr_block_select_workspace_bytes(d, 4) == 0
        assert hhr.hhr_block_attn_workspace_bytes(d, 4, 16) == 0


@pytest.mark.parametrize("call,names", [
    (append, ["k_new", "v_new", "start", "n_new", "pt", "k", "v", "ke", "ve"]),
    (read, ["k", "v", "ke", "ve", "pt", "start", "n", "ko", "vo"]),
    (paged, ["q", "k", "v", "pt", "seq", "out", "ws"]),
    (select, ["q", "seq", "pt", "mean", "blocks", "count", "ws"]),
    (block, ["q", "k", "v", "pt", "seq", "blocks", "count", "out", "ws"]),
])
def test_null_pointers(L, call, names):
    for n in names:
        assert call(L, _d(), **{n: None}) == INV, n


@pytest.mark.parametrize("call,names", [
    (append, ["k_new", "v_new", "k", "v", "ke", "ve", "mean"]),
    (read, ["k", "v", "ke", "ve", "ko", "vo"]),
    (paged, ["q", "k", "v", "out", "lse", "ws"]),
    (select, ["q", "mean", "ws"]),
    (block, ["q", "k", "v", "out", "lse", "ws"]),
])
def test_misaligned_pointers(L, call, names):
    for n in names:
        assert call(L, _d(), **{n: BAD}) == INV, n


def test_append_and_read_arguments(L):
    d = _d()
    assert append(L, d, stride=8 * 128 - 8) == INV      # rows that overlap
    assert append(L, d, stride=8 * 128 + 4) == INV      # rows that start off a 16-byte boundary
    assert append(L, d, stride=-8) == INV
    assert append(L, d, max_new=-1) == INV
    assert append(L, d, max_new=0) == hhr.HHR_OK
    assert read(L, d, max_n=-1) == INV
    assert read(L, d, max_n=0) == hhr.HHR_OK
    assert append(L, _d(page_size=1), max_new=(1 << 31) - 1) == UNS   # one page too many
    big = _d(page_size=256, n_phys_pages=1 << 21)       # 2^32 cache rows
    assert append(L, big) == UNS and read(L, big) == UNS


def test_paged_attention_arguments(L):
    d = _d()
    n = hhr.hhr_paged_attn_workspace_bytes(d)
    assert n > 0 and n % 256 == 0
    assert paged(L, d, n=n - 1) == WS
    assert paged(L, d, k_new=P) == INV and paged(L, d, v_new=P) == INV
    assert paged(L, d, k_new=BAD, v_new=P) == INV
    assert paged(L, d, ke=P) == INV and paged(L, d, ve=P) == INV
    assert paged(L, d, ke=BAD, ve=P) == INV
    assert paged(L, d, bf16=2) == INV
    for x in ("nan", "inf", "-inf", "3e38"):   # (also times log2 e)
        assert paged(L, d, scale=ctypes.c_float(float(x))) == INV
    assert paged(L, _d(select_per_head=1)) == INV       # nothing is selected
    assert paged(L, _d(n_q_heads=72)) == UNS            # 9 heads per KV head
    assert paged(L, _d(page_size=256, n_phys_pages=1 << 21)) == UNS
    # 65535 sequences of 2^23 keys: more units of work than an int counts.
    huge = _d(batch=65535, page_size=256, max_pages_per_seq=32768)
    assert paged(L, huge) == UNS and hhr.hhr_paged_attn_workspace_bytes(huge) == 0


def test_block_arguments(L):
    d = _d()
    n = hhr.hhr_block_select_workspace_bytes(d, 4)
    assert n >= 2 * 4 * 8 * 4096 * 4 and n % 256 == 0
    assert select(L, d, n=n - 1) == WS
    assert select(L, d, m=0) == INV and select(L, d, T=0) == INV
    assert select(L, d, opts=hhr.SelectOpts(-1, 0)) == INV
    assert select(L, d, opts=hhr.SelectOpts(10, 7)) == INV   # more than the 16 kept
    assert select(L, _d(n_q_heads=72)) == UNS
    assert select(L, d, T=1 << 27) == UNS
    n = hhr.hhr_block_attn_workspace_bytes(d, 4, 16)
    assert n > 0 and n % 256 == 0
    assert block(L, d, n=n - 1) == WS
    assert block(L, d, m=0) == INV and block(L, d, m=32769) == UNS
    assert block(L, d, T=0) == INV and block(L, d, T=1 << 27) == UNS
    assert block(L, d, ke=P) == INV and block(L, d, bf16=-1) == INV
    assert block(L, d, scale=ctypes.c_float(float("nan"))) == INV
    assert block(L, _d(page_size=256, n_phys_pages=1 << 21)) == UNS


# The binding: every call refuses host tensors and things that are no tensors, before anything
# else of theirs is used. (What it checks of CUDA tensors is tested in test_gpu_binding.py.)
HOST = torch.zeros(2, 4, 8, 128, dtype=torch.bfloat16)
BINDING_CALLS = {
    "hhr_append_kv8": lambda d, t: hhr.hhr_append_kv8(d, t, t, t, t, t, t, t, t, t),
    "hhr_read_kv8": lambda d, t: hhr.hhr_read_kv8(d, t, t, t, t, t, t, t, t, t),
    "hhr_paged_attn": lambda d, t: hhr.hhr_paged_attn(d, t, None, None, t, t, None, None, t, t,
                                                      0.1, t, t),
    "hhr_block_select": lambda d, t: hhr.hhr_block_select(d, t, t, t, t, t, 4, t, t, t),
    "hhr_block_attn": lambda d, t: hhr.hhr_block_attn(d, t, t, t, None, None, t, t, t, t, t, 0.1,
                                                      t, t),
}


@pytest.mark.parametrize("name", sorted(BINDING_CALLS))
def test_binding_refuses_what_is_no_cuda_tensor(L, name):
    call = BINDING_CALLS[name]
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(_d(), HOST)
    with pytest.raises(TypeError, match="torch tensor"):
        call(_d(), [1, 2])
    with pytest.raises(TypeError, match="dims"):
        call(b"not dims", HOST)
    with pytest.raises(TypeError):
        call(None, HOST)


def test_binding_module_is_required(L, monkeypatch, tmp_path):
    monkeypatch.setattr(hhr, "HERE", str(tmp_path))
    monkeypatch.setattr(hhr, "_binding", None)
    with pytest.raises(RuntimeError, match="missing"):
        hhr._native()


def test_binding_follows_a_reloaded_library(L, monkeypatch):
    """The module calls the library that hhr.lib() has loaded, also after it is loaded anew."""
    module = hhr._native()
    assert hhr.lib()._bound is module
    monkeypatch.setattr(hhr, "_lib", None)
    assert hhr._native() is module and hhr.lib()._bound is module


def test_binding_of_another_torch_is_rebuilt_and_refused(L, monkeypatch):
    """The module holds what it was built against; with another torch it is neither kept nor loaded."""
    assert build.binding_matches() and build.build_binding() is None
    assert hhr._native().built_for == build.binding_tag()
    started = []
    monkeypatch.setattr(build.subprocess, "Popen", lambda cmd, **kw: started.append(cmd))
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".1")
    assert not build.binding_matches()
    build.build_binding()
    assert len(started) == 1 and any(build.binding_tag() in x for x in started[0])
    monkeypatch.setattr(hhr, "_binding", None)
    with pytest.raises(RuntimeError, match="build it anew"):
        hhr._native()
