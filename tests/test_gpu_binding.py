"""What the compiled marshalling checks of CUDA tensors: types, layouts, sizes and strides, before
anything is launched."""
import math

import pytest
import torch

from hash_hierarchical_top_b200 import build, hhr
from page_helpers import D, Paged, status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def c():
    build.build()
    return Paged([40, 70], 2, 3, 16, True, seed=1)


def args_of(c, name):
    """A good call's tensors, by name, and the call."""
    B, G, Hq, T, m = 2, 2, 6, 3, 2
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    f32 = lambda *s: torch.zeros(*s, device="cuda")
    cache = dict(k=c.k, v=c.v, k_exp=c.k_exp, v_exp=c.v_exp)
    if name == "append":
        a = dict(k_new=bf(B, 1, G, D), v_new=bf(B, 1, G, D), start=i32(B), n_new=i32(B),
                 page_table=c.pt, **cache, block_mean=f32(c.n_phys, G, D))
        return a, lambda x: hhr.hhr_append_kv8(c.d, *x.values())
    if name == "read":
        a = dict(**cache, page_table=c.pt, start=i32(B), n=i32(B), k_out=bf(B, 4, G, D),
                 v_out=bf(B, 4, G, D))
        return a, lambda x: hhr.hhr_read_kv8(c.d, *x.values())
    if name == "paged":
        a = dict(q=bf(B, Hq, D), k_new=None, v_new=None, **cache, page_table=c.pt,
                 seq_len=c.seq_len, scale=0.1, out=f32(B, Hq, D),
                 workspace=torch.zeros(hhr.hhr_paged_attn_workspace_bytes(c.d), dtype=torch.uint8,
                                       device="cuda"), lse=f32(B, Hq))
        return a, lambda x: hhr.hhr_paged_attn(c.d, *x.values())
    if name == "select":
        a = dict(q=bf(B, T, Hq, D), seq_len=c.seq_len, q_pos=i32(B, T), page_table=c.pt,
                 block_mean=f32(c.n_phys, G, D), m_pages=m, out_blocks=i32(B, T, G, m),
                 out_count=i32(B, T, G),
                 workspace=torch.zeros(hhr.hhr_block_select_workspace_bytes(c.d, T),
                                       dtype=torch.uint8, device="cuda"))
        return a, lambda x: hhr.hhr_block_select(c.d, *x.values())
    a = dict(q=bf(B, T, Hq, D), **cache, page_table=c.pt, seq_len=c.seq_len, q_pos=i32(B, T),
             blocks=i32(B, T, G, m), block_count=i32(B, T, G), scale=0.1, out=f32(B, T, Hq, D),
             workspace=torch.zeros(hhr.hhr_block_attn_workspace_bytes(c.d, T, m),
                                   dtype=torch.uint8, device="cuda"), lse=f32(B, T, Hq))
    return a, lambda x: hhr.hhr_block_attn(c.d, *x.values())


@pytest.mark.parametrize("name", ["append", "read", "paged", "select", "block"])
def test_every_tensor_is_checked(c, name):
    a, call = args_of(c, name)
    call(a)
    status_ok()
    for key, t in a.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = torch.float64 if t.dtype != torch.float64 else torch.float32
        with pytest.raises(TypeError):
            call({**a, key: t.to(torch.float32).to(wrong)})
        with pytest.raises(ValueError):
            call({**a, key: t.cpu()})
        if key in ("workspace",):
            with pytest.raises(hhr.HHRError, match="WORKSPACE"):
                call({**a, key: t[:-256].clone()})
            continue
        with pytest.raises(ValueError):   # one row of the first dimension short
            call({**a, key: t[:-1].contiguous()})
        if t.dim() > 1 and key not in ("k_new", "v_new"):
            with pytest.raises(ValueError):
                call({**a, key: torch.stack([t, t], -1)[..., 0]})
    status_ok()


def test_none_where_a_tensor_is_needed(c):
    for name in ("append", "read", "paged", "select", "block"):
        a, call = args_of(c, name)
        for key, t in a.items():
            if not isinstance(t, torch.Tensor) or key in ("lse", "q_pos", "block_mean"):
                continue
            with pytest.raises((TypeError, ValueError, hhr.HHRError)):
                call({**a, key: None})
    status_ok()


def test_new_rows_may_be_slices_of_a_wider_row(c):
    a, call = args_of(c, "append")
    qkv = torch.zeros(2, 5, 10, D, dtype=torch.bfloat16, device="cuda")
    good = [(qkv[:, :, 6:8], qkv[:, :, 8:]), (qkv[:, 0, 6:8], qkv[:, 0, 8:]),
            (qkv[:, 4:, 6:8], qkv[:, 4:, 8:]), (qkv[:, :, :2].contiguous(),) * 2,
            (qkv[:, :0, :2],) * 2]
    for k, v in good:
        call({**a, "k_new": k, "v_new": v})
    k = qkv[:, :, 6:8]
    for bad in (k[:, 1:4], qkv[:, :, 6:10:2], qkv[:, :, 6:7], qkv[:1, :, 6:8], k.transpose(2, 3),
                qkv[:, 0, 0], k[:, ::2]):
        with pytest.raises(ValueError):
            call({**a, "k_new": bad, "v_new": bad})
    with pytest.raises(ValueError, match="same"):
        call({**a, "k_new": k, "v_new": k.contiguous()})
    status_ok()


def test_another_stream_is_taken(c):
    a, call = args_of(c, "paged")
    a["q"] = torch.randn(2, 6, D, device="cuda").bfloat16()
    call(a)
    ref = a["out"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        a["out"].zero_()
        torch.cuda.synchronize()
        hhr.hhr_paged_attn(c.d, *a.values(), stream=stream)
        s.synchronize()
        assert torch.equal(a["out"], ref)
    with pytest.raises(AttributeError):
        hhr.hhr_paged_attn(c.d, *a.values(), stream="x")
    status_ok()
    assert math.isfinite(float(ref.sum()))
