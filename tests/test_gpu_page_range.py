"""Attention over an 8-bit cache whose exponents lie far apart, and queries far from 1: legal inputs
that 16-bit matrix operands do not hold, against the float64 definition.

Tolerances are those of page_helpers, with a logit's error taken key by key (a key of negligible
weight may have a long, and so less exact, product): a weight w_j is off by w_j ds_j, and so
  |o - o_ref| <= sum_j w_j ds_j |v_j| + |o_ref| sum_j w_j ds_j + (2^-21 + sums) sum_j w_j |v_j|
                 + 2^-25 sum_j |v_j|     (weights normalised to a sum of 1, the last of them to a
                                          largest weight of 1, over their sum)
where the last term is what a weight loses below the matrix operands' range, relative to the largest.
"""
import math

import pytest
import torch

from hash_hierarchical_top_b200 import build, hhr
from page_helpers import D, Paged, check, status_ok

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)


def ref_rows(q, k, v, scale):
    """(o, lse, tolerances) of q [h, D] over rows k, v [n, D] in float64."""
    q, n = q.double(), len(k)
    s = scale * (q @ k.T)
    ds = 2.0 ** -19 * abs(scale) * (q.abs() @ k.abs().T) + 2.0 ** -22 * s.abs()
    top = s.amax(1, keepdim=True)
    w = torch.exp(s - top)
    total = w.sum(1, keepdim=True)
    o, lse = (w @ v) / total, (top + total.log())[:, 0]
    off = (w * ds).sum(1, keepdim=True) / total
    sums = (n / 128 + 64) * 2.0 ** -22
    tol = ((w * ds) @ v.abs() / total + o.abs() * off + (2.0 ** -21 + sums) * (w @ v.abs()) / total +
           2.0 ** -25 * v.abs().sum(0) / total)
    # fp32 results below 2^-126 have an absolute step of 2^-149.
    return o, lse, tol + 2.0 ** -146, off[:, 0] + sums + 2.0 ** -22 * lse.abs()


def run(c, q, path, scale=SCALE):
    """Outputs [h, D] and lse [h] per KV head of a single sequence, by a dense call or a list of all
    its pages."""
    out = torch.full((1, c.G * c.gs, D), math.nan, device="cuda")
    lse = torch.full((1, c.G * c.gs), math.nan, device="cuda")
    if path == "dense":
        ws = torch.full((hhr.hhr_paged_attn_workspace_bytes(c.d),), 0xff, dtype=torch.uint8, device="cuda")
        hhr.hhr_paged_attn(c.d, q, None, None, c.k, c.v, c.k_exp, c.v_exp, c.pt, c.seq_len, scale, out, ws,
                           lse=lse)
    else:
        n = -(-c.lens[0] // c.P)
        blocks = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, 1, c.G, n).contiguous()
        count = torch.full((1, 1, c.G), n, dtype=torch.int32, device="cuda")
        ws = torch.full((hhr.hhr_block_attn_workspace_bytes(c.d, 1, n),), 0xff, dtype=torch.uint8,
                        device="cuda")
        hhr.hhr_block_attn(c.d, q[:, None], c.k, c.v, c.k_exp, c.v_exp, c.pt, c.seq_len, None, blocks, count,
                           scale, out[:, None], ws, lse=lse[:, None])
    status_ok()
    return out[0], lse[0]


def check_all(c, q, out, lse, scale=SCALE):
    pos = torch.arange(c.lens[0], device="cuda")
    for g in range(c.G):
        h = slice(g * c.gs, (g + 1) * c.gs)
        o, l, to, tl = ref_rows(q[0, h], c.rows("k", 0, g, pos), c.rows("v", 0, g, pos), scale)
        check(out[h], o, to, f"KV head {g}")
        check(lse[h], l, tl, f"KV head {g} lse")


def put(c, name, pos, values, exp):
    """Row `pos` of sequence 0, all KV heads: e4m3 bytes {channel: byte}, zeros elsewhere."""
    phys, slot = int(c.pt[0, pos // c.P]), pos % c.P
    x, e = getattr(c, name), getattr(c, name + "_exp")
    x[phys, :, slot] = 0
    for ch, byte in values.items():
        x[phys, :, slot, ch] = byte
    e[phys, :, slot] = exp


def against(c, q, pos, size):
    """Key row `pos` becomes -size times the sum of its group's queries: little weight everywhere."""
    from page_helpers import quantise_ref
    phys, slot = int(c.pt[0, pos // c.P]), pos % c.P
    x = -size * q[0].float().reshape(c.G, c.gs, D).sum(1)
    b, e = quantise_ref(x.bfloat16())
    c.k[phys, :, slot], c.k_exp[phys, :, slot] = b.cuda(), e.cuda()


# Lengths that a cluster per row takes, and ones that are split evenly over all CTAs.
PATHS = [("dense", 600), ("dense", 9001), ("list", 600), ("list", 20000)]


@pytest.mark.parametrize("gap", [0, 8, 13, 14, 15, 17, 20, 24, 30, 34, 40, 60, 90, 126])
@pytest.mark.parametrize("negligible", [True, False])
@pytest.mark.parametrize("gs", [2, 5])
@pytest.mark.parametrize("path,n", PATHS)
def test_value_rows_of_larger_exponents(path, n, gs, negligible, gap):
    """Two value rows far larger than the others, in one channel only, one of them among the first
    keys: the other channels are the other keys' sums, whatever the large rows weigh."""
    build.build()
    c = Paged([n], 1, gs, 32, True, seed=100 + gap)
    q = c.queries(1)
    for pos in (1, n - 70):
        if negligible:
            against(c, q, pos, 3.0)
        put(c, "v", pos, {9: 0x7e}, 120 + gap)            # 448 * 2^(gap - 7)
    check_all(c, q, *run(c, q, path))


@pytest.mark.parametrize("path,n", PATHS)
@pytest.mark.parametrize("gap", [12, 14, 16, 25, 40, 105])
def test_value_rows_of_smaller_exponents(path, n, gap):
    """One key that nearly takes all, whose value row is far smaller than the others; in channels
    that the others leave empty it is all there is."""
    build.build()
    c = Paged([n], 2, 4, 16, True, seed=200 + gap)
    c.v[..., 64:] = torch.where(c.v_exp[..., None] == 255, c.v[..., 64:], torch.zeros_like(c.v[..., 64:]))
    q = c.queries(1)
    against(c, q, 37, -0.5)
    put(c, "v", 37, {ch: 0x3a + ch % 7 for ch in range(D)}, max(10, 120 - gap))
    check_all(c, q, *run(c, q, path))


@pytest.mark.parametrize("weight", [3.0, 0.0])
@pytest.mark.parametrize("path,n", PATHS)
def test_an_infinite_value_acts_on_its_channel_only(path, n, weight):
    """A value row with an infinity, as the append quantises it: 448 * 2^119 in that channel."""
    build.build()
    c = Paged([n], 2, 4, 32, True, seed=300)
    q = c.queries(1)
    new = torch.randn(1, 1, 2, D, device="cuda").bfloat16()
    new[..., 77] = math.inf
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    hhr.hhr_append_kv8(c.d, new.clone().nan_to_num(1.0, 1.0), new, i32(n - 1), i32(1), c.pt, c.k, c.v,
                       c.k_exp, c.v_exp)
    if weight:
        against(c, q, n - 1, weight)
    out, lse = run(c, q, path)
    check_all(c, q, out, lse)
    assert (out[:, 77] > 1e6).all() and (out[:, :77].abs() < 10).all()


@pytest.mark.parametrize("path,n", PATHS)
def test_value_rows_of_zeros(path, n):
    """Rows of zeros (the smallest exponent byte, zeros of both signs) among ordinary ones, and one
    row under the same byte that is not zero, in a channel of its own."""
    build.build()
    c = Paged([n], 1, 4, 32, True, seed=310)
    q = c.queries(1)
    for pos in range(0, n, 5):
        put(c, "v", pos, {3: 0x80}, 10)
    check_all(c, q, *run(c, q, path))
    c.v[..., 5] = torch.where(c.v_exp == 255, c.v[..., 5], torch.zeros_like(c.v[..., 5]))
    put(c, "v", 300, {5: 0x7e}, 10)
    out, lse = run(c, q, path)
    check_all(c, q, out, lse)
    assert (out[:, 5] > 0).all()


@pytest.mark.parametrize("gs", [3, 8])
@pytest.mark.parametrize("path,n", PATHS)
@pytest.mark.parametrize("qs,ks", [(-60, 58), (-100, 100), (-112, 112), (-118, 116), (-124, 117), (100, -100),
                                   (120, -115), (125, -117), (-60, 118)])
def test_queries_and_keys_of_any_size(qs, ks, path, n, gs):
    """Query times key in fp32's range, wherever its factors lie."""
    build.build()
    c = Paged([n], 1, gs, 32, True, seed=400, scale=2.0 ** ks)
    q = (c.queries(1).float() * 2.0 ** qs).bfloat16()
    # (Sizes whose logits pass what softmax tells apart are scaled down to it.)
    scale = SCALE * 2.0 ** -max(0, qs + ks - 1)
    out, lse = run(c, q, path, scale)
    check_all(c, q, out, lse, scale)


@pytest.mark.parametrize("path,n", PATHS)
@pytest.mark.parametrize("spread", [20, 30, 32, 40, 100])
def test_query_channels_of_very_different_sizes(path, n, spread):
    """The largest query channel meets keys that are 0 there: the small channels decide."""
    build.build()
    c = Paged([n], 1, 4, 32, True, seed=500 + spread)
    q = c.queries(1)
    q[:, :, 11] = 1.5 * 2.0 ** spread
    c.k[..., 11] = torch.where(c.k_exp == 255, c.k[..., 11], torch.zeros_like(c.k[..., 11]))
    check_all(c, q, *run(c, q, path))


@pytest.mark.parametrize("kind", ["zero queries", "one zero query", "one infinite key byte"])
def test_zero_queries_and_single_large_keys(kind):
    build.build()
    c = Paged([700], 1, 4, 32, True, seed=600)
    q = c.queries(1)
    if kind == "zero queries":
        q.zero_()
    elif kind == "one zero query":
        q[:, 2] = 0
    else:
        q[..., 4] = 0
        put(c, "k", 123, {4: 0x7e}, 246)                  # 448 * 2^119 where every query is 0
    check_all(c, q, *run(c, q, "dense"))


@pytest.mark.parametrize("path,n", PATHS)
def test_nan_and_infinite_queries_act_on_their_heads_only(path, n):
    """Beside an ordinary cache, and beside one that the wide range is needed for."""
    build.build()
    for far in (False, True):
        c = Paged([n], 1, 4, 32, True, seed=700)
        q = c.queries(1)
        q[0, 1, 5] = math.nan
        q[0, 2, 6] = math.inf
        if far:
            put(c, "v", 40, {9: 0x7e}, 200)
        c.k[..., 6] = torch.where(c.k_exp == 255, c.k[..., 6], torch.full_like(c.k[..., 6], 0x38))
        out, lse = run(c, q, path)
        assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
        keep = [0, 3]
        pos = torch.arange(n, device="cuda")
        o, l, to, tl = ref_rows(q[0, keep], c.rows("k", 0, 0, pos), c.rows("v", 0, 0, pos), SCALE)
        check(out[keep], o, to, "rest")
        check(lse[keep], l, tl, "rest lse")


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("n", [600, 9001])
@pytest.mark.parametrize("qs,ks,scale", [(60, 58, 0.0), (60, 58, -0.0), (100, 24, 0.0), (60, 58, 2.0 ** -128),
                                         (60, 58, -2.0 ** -127), (20, -19, 1.0)])
def test_scales_of_zero_and_below_the_normal_range(qs, ks, scale, n, kv8):
    """A scale of 0 is the plain mean, however large the products are; one below 2^-126 is taken as it is."""
    build.build()
    c = Paged([n], 1, 4, 32, kv8, seed=800, scale=2.0 ** ks)
    q = (c.queries(1).float() * 2.0 ** qs).bfloat16()
    out, lse = run(c, q, "dense", scale)
    check_all(c, q, out, lse, scale)


@pytest.mark.parametrize("kv8", [False, True])
def test_a_scale_of_zero_keeps_infinite_and_nan_queries(kv8):
    build.build()
    c = Paged([300], 1, 4, 32, kv8, seed=801)
    q = c.queries(1)
    q[0, 1, 5], q[0, 2, 6] = math.nan, -math.inf
    out, lse = run(c, q, "dense", 0.0)
    assert torch.isnan(out[1:3]).all() and torch.isfinite(out[[0, 3]]).all()


@pytest.mark.parametrize("pages", [8, 600])
def test_many_sequences_with_far_rows_new_ones_among_them(pages):
    """A ragged batch of more sequences than a warp scans, some with far rows, some with a far new row
    that the call writes; captured once and replayed over other rows."""
    build.build()
    P, G, gs, B = 16, 2, 4, 41
    lens = [(97 * i) % (5 * P) for i in range(B)]
    lens[7], lens[30] = pages * P, pages * P - 3
    c = Paged(lens, G, gs, P, True, seed=900, extra_cols=0)
    q = c.queries(B)
    kn, vn = (torch.randn(B, G, D, device="cuda").bfloat16() for _ in "kv")
    vn[3::5, :, 9] = math.inf
    vn[4::5, 0, 100] = 2.0 ** 60
    for b in (7, 11, 30):
        phys, slot = int(c.pt[b, 1]), 5
        c.v[phys, 0, slot] = 0
        c.v[phys, 0, slot, 77], c.v_exp[phys, 0, slot] = 0x7e, 190
    out = torch.full((B, G * gs, D), math.nan, device="cuda")
    lse = torch.full((B, G * gs), math.nan, device="cuda")
    ws = torch.full((hhr.hhr_paged_attn_workspace_bytes(c.d),), 0xff, dtype=torch.uint8, device="cuda")

    def call():
        hhr.hhr_paged_attn(c.d, q, kn, vn, c.k, c.v, c.k_exp, c.v_exp, c.pt, c.seq_len, SCALE, out, ws, lse=lse)

    def verify():
        status_ok()
        for b, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            for g in range(G):
                h = slice(g * gs, (g + 1) * gs)
                if n == 0:
                    assert (out[b, h] == 0).all() and (lse[b, h] == -math.inf).all()
                    continue
                o, l, to, tl = ref_rows(q[b, h], c.rows("k", b, g, pos), c.rows("v", b, g, pos), SCALE)
                check(out[b, h], o, to, f"sequence {b}, KV head {g}")
                check(lse[b, h], l, tl, f"sequence {b}, KV head {g} lse")

    call()
    verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for far in (0, 1):
        vn.normal_()
        if far:
            vn[::3, 1, 64] = 2.0 ** 90
        q.normal_()
        out.fill_(math.nan)
        graph.replay()
        verify()


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("P,m", [(16, 5), (128, 40)])
def test_a_chunk_of_queries_over_far_rows(P, m, per_head):
    """Lists of several queries, causal, some of which name a page with a far row."""
    build.build()
    lens, G, gs, T = [9000, 400], 2, 4, 3
    c = Paged(lens, G, gs, P, True, seed=910)
    c.d.select_per_head = int(per_head)
    rows = G * gs if per_head else G
    q = c.queries(2, T)
    for b, page in ((0, 2), (0, 3000 // P), (1, 0)):
        phys = int(c.pt[b, page])
        c.v[phys, :, 3] = 0
        c.v[phys, :, 3, 50], c.v_exp[phys, :, 3] = 0x7e, 200
    gen = torch.Generator(device="cuda").manual_seed(911)
    pages = torch.tensor([-(-n // P) for n in lens], device="cuda")
    blocks = (torch.rand(2, T, rows, m, generator=gen, device="cuda") * pages[:, None, None, None]).int()
    blocks[:, 0, :, 1] = 2 if P == 16 else 0
    count = torch.full((2, T, rows), m, dtype=torch.int32, device="cuda")
    q_pos = torch.tensor([[n - 300, n - 2, n + 5] for n in lens], dtype=torch.int32, device="cuda")
    out, lse = torch.full(q.shape, math.nan, device="cuda"), torch.full(q.shape[:-1], math.nan, device="cuda")
    ws = torch.full((hhr.hhr_block_attn_workspace_bytes(c.d, T, m),), 0xff, dtype=torch.uint8, device="cuda")
    hhr.hhr_block_attn(c.d, q, c.k, c.v, c.k_exp, c.v_exp, c.pt, c.seq_len, q_pos, blocks, count, SCALE, out, ws,
                       lse=lse)
    status_ok()
    per = G * gs // rows
    for b, n in enumerate(lens):
        for t in range(T):
            for r in range(rows):
                at = (blocks[b, t, r].long()[:, None] * P + torch.arange(P, device="cuda")).reshape(-1)
                at = at[at < min(n, int(q_pos[b, t]) + 1)]
                g, h = r * G // rows, slice(r * per, (r + 1) * per)
                o, l, to, tl = ref_rows(q[b, t, h], c.rows("k", b, g, at), c.rows("v", b, g, at), SCALE)
                check(out[b, t, h], o, to, f"sequence {b}, query {t}, row {r}")
                check(lse[b, t, h], l, tl, f"sequence {b}, query {t}, row {r} lse")
