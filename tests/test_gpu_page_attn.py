"""Dense paged attention and block-sparse attention on the GPU against float64 references, from
bf16 and 8-bit caches whose unused slots hold NaNs."""
import math

import pytest
import torch

from hash_hierarchical_top_b200 import build, hhr
from page_helpers import D, Paged, check_rows, quantise_ref, status_ok, values_of

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)


def dense(c, q, out_dtype=torch.float32, k_new=None, v_new=None, scale=SCALE, ws=None):
    out = torch.full(q.shape, math.nan, dtype=out_dtype, device="cuda")
    lse = torch.full(q.shape[:-1], math.nan, device="cuda")
    if ws is None:
        ws = torch.full((hhr.hhr_paged_attn_workspace_bytes(c.d),), 0xff, dtype=torch.uint8,
                        device="cuda")
    hhr.hhr_paged_attn(c.d, q, k_new, v_new, c.k, c.v, c.k_exp, c.v_exp, c.pt, c.seq_len, scale,
                       out, ws, lse=lse)
    return out, lse


def check_dense(c, q, out, lse, scale=SCALE):
    for b, n in enumerate(c.lens):
        pos = torch.arange(n, device="cuda")
        for g in range(c.G):
            h = slice(g * c.gs, (g + 1) * c.gs)
            check_rows(out[b, h], lse[b, h], q[b, h], c.rows("k", b, g, pos),
                       c.rows("v", b, g, pos), scale, f"sequence {b}, KV head {g}")


SHAPES = [  # lengths, KV heads, heads per KV head, page size
    ([1], 1, 1, 1),
    ([2, 1, 0, 3], 2, 8, 16),
    ([517], 8, 4, 32),
    ([127, 128, 129, 0, 255, 257], 3, 5, 32),
    ([1000, 31], 1, 7, 17),
    ([4096], 1, 1, 64),
    ([5000, 1, 300], 2, 3, 5),
    ([777, 2049], 4, 2, 256),
    ([300], 2, 6, 1),
    ([9001], 2, 8, 100),
]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("lens,G,gs,P", SHAPES)
def test_dense(lens, G, gs, P, kv8, out_dtype):
    build.build()
    c = Paged(lens, G, gs, P, kv8, seed=len(lens) + P)
    q = c.queries(len(lens))
    out, lse = dense(c, q, out_dtype)
    status_ok()
    check_dense(c, q, out, lse)


@pytest.mark.parametrize("kv8", [False, True])
def test_dense_many_ragged_sequences(kv8):
    """More sequences than threads of a CTA, most of them short, one long."""
    build.build()
    lens = [(37 * i) % 90 for i in range(300)]
    lens[211] = 20000
    c = Paged(lens, 1, 4, 16, kv8, seed=8)
    q = c.queries(300)
    out, lse = dense(c, q)
    status_ok()
    check_dense(c, q, out, lse)


@pytest.mark.parametrize("kv8", [False, True])
def test_dense_many_sequences_write_their_newest_rows(kv8):
    build.build()
    lens = [(29 * i) % 200 for i in range(100)]
    c = Paged(lens, 2, 2, 16, kv8, seed=9)
    new = [torch.randn(100, 2, D, device="cuda").bfloat16() for _ in "kv"]
    q = c.queries(100)
    out, lse = dense(c, q, k_new=new[0], v_new=new[1])
    status_ok()
    for b, n in enumerate(lens):
        if n:
            for name, x in zip("kv", new):
                got = torch.stack([c.rows(name, b, g, torch.tensor([n - 1], device="cuda"))[0] for g in range(2)])
                # The 8-bit row: half a step of 2^-4, or 2^(e - 10) below the smallest normal number.
                x = x[b].double()
                tol = (2.0 ** -4 * x.abs()).clamp(min=float(x.abs().max()) / 224 * 2.0 ** -10) if kv8 else 0
                assert ((got - x).abs() <= tol).all()
    check_dense(c, q, out, lse)


@pytest.mark.parametrize("kv8", [False, True])
def test_dense_long_sequence_peaked_and_flat(kv8):
    """64K keys split over every CTA: a query that one key dominates, and a nearly flat one whose
    65536 weights are all of the same size."""
    build.build()
    n = 65536
    c = Paged([n, n], 1, 2, 32, kv8, seed=3)
    q = c.queries(2)
    q[1] *= 0.01
    k = c.rows("k", 0, 0, torch.arange(n, device="cuda"))
    q[0, 0] = (k[54321] * 3).bfloat16()
    out, lse = dense(c, q)
    status_ok()
    check_dense(c, q, out, lse)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("gs", [3, 7])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_dense_scales(scale, gs, kv8):
    """A scale of 0 (the plain mean), a negative and a large one (one key takes nearly all)."""
    build.build()
    c = Paged([700, 1, 0], 2, gs, 32, kv8, seed=13)
    q = c.queries(3)
    out, lse = dense(c, q, scale=scale)
    status_ok()
    check_dense(c, q, out, lse, scale)


@pytest.mark.parametrize("kv8", [False, True])
def test_dense_large_and_small_magnitudes(kv8):
    """Queries and keys far from 1, with one key or value row at another exponent than the rest."""
    build.build()
    for qs, ks in ((2.0 ** 40, 2.0 ** -42), (2.0 ** -60, 2.0 ** 58), (8.0, 4.0)):
        c = Paged([600], 2, 4, 32, kv8, seed=11, scale=ks)
        q = (c.queries(1).float() * qs).bfloat16()
        if kv8:
            phys = int(c.pt[0, 3])
            c.v_exp[phys, :, 7] = 150            # 2^23 times the others' size
            c.v_exp[phys, :, 8] = 60
            c.k_exp[phys, :, 9] = 20
        out, lse = dense(c, q)
        status_ok()
        check_dense(c, q, out, lse)


def test_tiny_values_of_an_8bit_cache():
    """Value rows at the smallest exponents (their values are 2^-126 times whole numbers)."""
    build.build()
    c = Paged([200], 1, 2, 32, True, seed=12)
    c.v_exp[c.v_exp != 255] = 10
    q = c.queries(1)
    out, lse = dense(c, q)
    status_ok()
    o = torch.zeros(2, D, dtype=torch.float64, device="cuda")
    pos = torch.arange(200, device="cuda")
    from page_helpers import attend_ref
    o, _, tol, _ = attend_ref(q[0], c.rows("k", 0, 0, pos), c.rows("v", 0, 0, pos), SCALE)
    # fp32 results below 2^-126 have an absolute step of 2^-149: a few of them.
    assert ((out[0].double() - o).abs() <= tol + 2.0 ** -146).all() and (out != 0).any()


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("lens,G,gs,P", SHAPES)
def test_dense_writes_the_newest_row(lens, G, gs, P, kv8):
    """k_new, v_new land in the newest position and nowhere else, and are attended to."""
    build.build()
    c = Paged(lens, G, gs, P, kv8, seed=21 + P)
    B = len(lens)
    k_new = torch.randn(B, G, D, device="cuda").bfloat16() * 3
    v_new = torch.randn(B, G, D, device="cuda").bfloat16() * 2
    want = [x.clone() if x is not None else None for x in (c.k, c.v, c.k_exp, c.v_exp)]
    for b, n in enumerate(lens):
        if n == 0:
            continue
        phys, slot = int(c.pt[b, (n - 1) // P]), (n - 1) % P
        for i, x in ((0, k_new), (1, v_new)):
            if kv8:
                y, e = quantise_ref(x[b])
                want[i][phys, :, slot], want[i + 2][phys, :, slot] = y.cuda(), e.cuda()
            else:
                want[i][phys, :, slot] = x[b]
    q = c.queries(B)
    out, lse = dense(c, q, k_new=k_new, v_new=v_new)
    status_ok()
    for got, ref in zip((c.k, c.v, c.k_exp, c.v_exp), want):
        if ref is not None:
            bits = torch.uint8 if kv8 else torch.int16
            assert torch.equal(got.view(bits), ref.view(bits))
    check_dense(c, q, out, lse)


def blocks_of(c, T, rows, m, seed, pos):
    """Random block lists: unsorted, one block twice, some lists empty or shorter than m."""
    gen = torch.Generator().manual_seed(seed)
    B = len(c.lens)
    blocks = torch.full((B, T, rows, m), 1 << 20, dtype=torch.int32)  # past the count: anything
    count = torch.zeros(B, T, rows, dtype=torch.int32)
    for b in range(B):
        n_pages = -(-c.lens[b] // c.P)
        for t in range(T):
            for r in range(rows):
                k = int(torch.randint(0, m + 1, (1,), generator=gen)) if n_pages else 0
                pick = torch.randint(0, max(n_pages, 1), (k,), generator=gen)
                if k >= 2:
                    pick[k // 2] = pick[0]
                blocks[b, t, r, :k] = pick.int()
                count[b, t, r] = k
    return blocks.cuda(), count.cuda()


def sparse(c, q, blocks, count, q_pos, out_dtype=torch.float32):
    out = torch.full(q.shape, math.nan, dtype=out_dtype, device="cuda")
    lse = torch.full(q.shape[:-1], math.nan, device="cuda")
    ws = torch.full((hhr.hhr_block_attn_workspace_bytes(c.d, q.shape[1], blocks.shape[-1]),), 0xff,
                    dtype=torch.uint8, device="cuda")
    hhr.hhr_block_attn(c.d, q, c.k, c.v, c.k_exp, c.v_exp, c.pt, c.seq_len, q_pos, blocks, count,
                       SCALE, out, ws, lse=lse)
    return out, lse


def check_sparse(c, q, blocks, count, q_pos, out, lse):
    rows = blocks.shape[2]
    gs = c.G * c.gs // rows
    for b, n in enumerate(c.lens):
        for t in range(q.shape[1]):
            limit = n if q_pos is None else min(n, int(q_pos[b, t]) + 1)
            for r in range(rows):
                chosen = blocks[b, t, r, :int(count[b, t, r])].long()
                pos = (chosen[:, None] * c.P + torch.arange(c.P, device="cuda")).reshape(-1)
                pos = pos[pos < limit]
                h, g = slice(r * gs, (r + 1) * gs), r * c.G // rows
                check_rows(out[b, t, h], lse[b, t, h], q[b, t, h], c.rows("k", b, g, pos),
                           c.rows("v", b, g, pos), SCALE, f"sequence {b}, query {t}, row {r}")


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("lens,G,gs,P,T,m,causal", [
    ([1], 1, 1, 1, 1, 1, False),
    ([700, 0, 33], 2, 4, 32, 1, 5, False),
    ([700, 90, 33], 2, 3, 17, 4, 3, True),
    ([2000], 8, 4, 128, 16, 4, True),
    ([4000, 3999], 1, 8, 64, 1, 40, False),
    ([513], 3, 5, 5, 9, 60, True),
    ([300, 260], 2, 7, 256, 2, 2, True),
])
def test_blocks(lens, G, gs, P, T, m, causal, kv8, per_head):
    build.build()
    c = Paged(lens, G, gs, P, kv8, seed=31 + P)
    c.d.select_per_head = int(per_head)
    rows = G * gs if per_head else G
    q = c.queries(len(lens), T)
    # Positions from before the first key to past the last.
    q_pos = (torch.linspace(-1, max(lens) + 3, T, device="cuda").int().expand(len(lens), T)
             .contiguous() if causal else None)
    blocks, count = blocks_of(c, T, rows, m, 7 * P + T, q_pos)
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = sparse(c, q, blocks, count, q_pos, dtype)
        status_ok()
        check_sparse(c, q, blocks, count, q_pos, out, lse)


def test_every_block_listed_equals_dense_attention():
    """All pages listed in order: the same sums as the dense call, up to their split."""
    build.build()
    for kv8 in (False, True):
        c = Paged([3001], 2, 4, 32, kv8, seed=41)
        q = c.queries(1)
        n = -(-3001 // 32)
        blocks = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, 1, 2, n).contiguous()
        count = torch.full((1, 1, 2), n, dtype=torch.int32, device="cuda")
        out, lse = sparse(c, q[:, None], blocks, count, None)
        status_ok()
        check_dense(c, q, out[:, 0], lse[:, 0])


def test_joining_two_halves_by_their_lse():
    """Outputs over disjoint block sets, joined by their log-sums, are those over the union."""
    build.build()
    c = Paged([2048], 2, 4, 32, False, seed=51)
    q = c.queries(1, 1)
    parts = []
    for lo, hi in ((0, 20), (20, 64), (0, 64)):
        blocks = torch.arange(lo, hi, dtype=torch.int32, device="cuda").expand(1, 1, 2, hi - lo)
        count = torch.full((1, 1, 2), hi - lo, dtype=torch.int32, device="cuda")
        parts.append(sparse(c, q, blocks.contiguous(), count, None))
    status_ok()
    (o1, l1), (o2, l2), (o, l) = parts
    both = torch.logaddexp(l1, l2)
    joined = o1 * (l1 - both).exp()[..., None] + o2 * (l2 - both).exp()[..., None]
    check_dense(c, q[:, 0], joined[:, 0], both[:, 0])
    check_dense(c, q[:, 0], o[:, 0], l[:, 0])


def test_equal_inputs_give_equal_bits_on_any_stream_and_in_a_graph():
    build.build()
    c = Paged([9000, 77, 3000], 4, 4, 32, True, seed=61)
    q = c.queries(3)
    out, lse = dense(c, q)
    ref = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, _ = dense(c, q)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, ref)
    ws = torch.empty(hhr.hhr_paged_attn_workspace_bytes(c.d), dtype=torch.uint8, device="cuda")
    got, l2 = torch.empty_like(out), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hhr.hhr_paged_attn(c.d, q, None, None, c.k, c.v, c.k_exp, c.v_exp, c.pt, c.seq_len, SCALE,
                           got, ws, lse=l2)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, ref) and torch.equal(l2, lse)
    # Other lengths and queries through the same graph: nothing of the first call is kept.
    c.lens = [1, 5000, 0]
    c.pt[1, :] = c.pt[0, :]
    c.seq_len.copy_(torch.tensor(c.lens))
    q.copy_(c.queries(3))
    graph.replay()
    status_ok()
    check_dense(c, q, got, l2)


def test_bad_pages_and_blocks_are_skipped_and_flagged():
    build.build()
    for kv8 in (False, True):
        c = Paged([200, 200], 1, 2, 32, kv8, seed=71)
        q = c.queries(2)
        good = c.pt.clone()
        c.pt[0, 2] = c.n_phys + 5
        c.pt[1, 0] = -3
        out, lse = dense(c, q)
        torch.cuda.synchronize()
        assert hhr.hhr_read_device_status() == (hhr.HHR_ERR_DEVICE_STATUS, 1)
        bad, c.pt = c.pt, good
        for b, skip in ((0, 2), (1, 0)):
            pos = torch.arange(200, device="cuda")
            pos = pos[pos // 32 != skip]
            check_rows(out[b], lse[b], q[b], c.rows("k", b, 0, pos), c.rows("v", b, 0, pos), SCALE, "skip")
        # A length beyond the page table is clipped.
        c.seq_len[1] = c.maxp * 32 + 1
        c.pt[1, -1] = c.pt[0, 0]
        c.pt[1, -2] = c.pt[0, 1]
        dense(c, q)
        torch.cuda.synchronize()
        assert hhr.hhr_read_device_status() == (hhr.HHR_ERR_DEVICE_STATUS, 2)
        c.seq_len[1] = 200
        blocks = torch.tensor([[[[1, -1, 3]]], [[[c.maxp, 0, 2]]]], dtype=torch.int32, device="cuda")
        count = torch.full((2, 1, 1), 3, dtype=torch.int32, device="cuda")
        out, lse = sparse(c, q[:, None], blocks, count, None)
        torch.cuda.synchronize()
        assert hhr.hhr_read_device_status() == (hhr.HHR_ERR_DEVICE_STATUS, 2)
        for b, keep in ((0, (1, 3)), (1, (0, 2))):
            pos = torch.cat([torch.arange(32 * p, 32 * p + 32, device="cuda") for p in keep])
            check_rows(out[b, 0], lse[b, 0], q[b], c.rows("k", b, 0, pos), c.rows("v", b, 0, pos), SCALE, "skip")


@pytest.mark.parametrize("kv8", [False, True])
def test_nan_and_infinite_keys_act_on_their_heads_only(kv8):
    """A NaN in a key makes its row NaN and no other; a value's NaN likewise its channel."""
    build.build()
    c = Paged([300, 300], 2, 2, 32, kv8, seed=81)
    phys = int(c.pt[0, 1])
    if kv8:
        c.k[phys, 0, 3, 5] = 0x7f
        c.v[phys, 1, 3, 9] = 0x7f
    else:
        c.k[phys, 0, 3, 5] = math.nan
        c.v[phys, 1, 3, 9] = math.nan
    q = c.queries(2)
    out, lse = dense(c, q)
    status_ok()
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert torch.isnan(out[0, 2:, 9]).all()
    clean = torch.arange(D, device="cuda") != 9
    assert torch.isfinite(out[0, 2:][:, clean]).all() and torch.isfinite(out[1]).all()
    assert torch.isfinite(lse[0, 2:]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("pages", [3, 400])
@pytest.mark.parametrize("kv8", [False, True])
def test_a_new_row_without_a_page_is_not_written(kv8, pages):
    """A length past the page table, or a newest page that is out of range: flagged, and no row of
    the cache is touched (by a cluster's kernel and by the even shares')."""
    build.build()
    n = pages * 16
    c = Paged([n, n], 1, 2, 16, kv8, seed=83, extra_cols=0)
    assert c.maxp * 16 == n
    new = torch.randn(2, 1, D, device="cuda").bfloat16()
    before = [x.clone() for x in (c.k, c.v, c.k_exp, c.v_exp) if x is not None]
    q = c.queries(2)
    for page, bits in ((c.n_phys, 1), (-1, 1), (-(1 << 31), 1)):
        good = int(c.pt[0, -1])
        c.pt[0, -1] = page
        c.seq_len[1] = n + 1                               # sequence 1 has no page for it
        dense(c, q, k_new=new, v_new=new)
        torch.cuda.synchronize()
        assert hhr.hhr_read_device_status() == (hhr.HHR_ERR_DEVICE_STATUS, bits | 2)
        c.pt[0, -1] = good
        for x, y in zip([x for x in (c.k, c.v, c.k_exp, c.v_exp) if x is not None], before):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_extreme_list_entries_are_flagged():
    build.build()
    c = Paged([200], 1, 2, 32, False, seed=87)
    q = c.queries(1)
    for entry in (-(1 << 31), (1 << 31) - 1, -1):
        blocks = torch.tensor([[[[entry, 2, 5]]]], dtype=torch.int32, device="cuda")
        count = torch.full((1, 1, 1), 9, dtype=torch.int32, device="cuda")   # clipped to 3
        out, lse = sparse(c, q[:, None], blocks, count, None)
        torch.cuda.synchronize()
        assert hhr.hhr_read_device_status() == (hhr.HHR_ERR_DEVICE_STATUS, 2)
        pos = torch.cat([torch.arange(64, 96), torch.arange(160, 192)]).cuda()
        check_rows(out[0, 0], lse[0, 0], q[0], c.rows("k", 0, 0, pos), c.rows("v", 0, 0, pos), SCALE, "rest")


def test_infinite_keys_of_a_bf16_cache():
    """A key that is +-infinite in a channel: heads whose logit is -inf leave it out, heads whose
    logit is +inf (or NaN) become NaN, as the formula says."""
    build.build()
    c = Paged([300], 1, 4, 32, False, seed=82)
    phys = int(c.pt[0, 5])
    c.k[phys, 0, 9, 4] = math.inf                       # position 169
    q = c.queries(1)
    q[0, :, 4] = torch.tensor([-1.0, 2.0, -0.5, 0.0]).bfloat16().cuda()
    out, lse = dense(c, q)
    status_ok()
    pos = torch.arange(300, device="cuda")
    pos = pos[pos != 169]
    k, v = c.rows("k", 0, 0, pos), c.rows("v", 0, 0, pos)
    for h in (0, 2):
        check_rows(out[0, h:h + 1], lse[0, h:h + 1], q[0, h:h + 1], k, v, SCALE, f"head {h}")
    assert torch.isnan(out[0, 1]).all() and torch.isnan(out[0, 3]).all()


def test_two_calls_at_once_on_two_streams():
    """Calls that overlap, each with its own workspace, do not disturb one another."""
    build.build()
    a, b = Paged([20000], 2, 4, 32, False, seed=84), Paged([15000, 300], 2, 4, 16, True, seed=85)
    qa, qb = a.queries(1), b.queries(2)
    ra, rb = dense(a, qa)[0].clone(), dense(b, qb)[0].clone()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s):
            got.append((dense(a, qa)[0], ra))
        with torch.cuda.stream(t):
            got.append((dense(b, qb)[0], rb))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)
    status_ok()


def test_a_call_sees_what_the_kernels_before_it_wrote():
    """Every call's first kernel is placed while the one before it still runs: its inputs (written
    just before, by other kernels of the stream) must nevertheless be the new ones."""
    build.build()
    c = Paged([3000, 500], 2, 4, 32, True, seed=86)
    big = torch.randn(1 << 24, device="cuda")
    q, outs, qs = c.queries(2), [], []
    ws = torch.empty(hhr.hhr_paged_attn_workspace_bytes(c.d), dtype=torch.uint8, device="cuda")
    for i in range(8):
        new = c.queries(2)
        big.mul_(1.0001)                                # keeps the GPU busy
        q.copy_(new)
        outs.append(dense(c, q, ws=ws))
        qs.append(new)
    status_ok()
    for new, (out, lse) in zip(qs, outs):
        check_dense(c, new, out, lse)


def test_8bit_cache_past_4_gigabytes():
    """Rows whose byte offsets pass 32 bits: appended, read back, attended to (dense and listed)."""
    build.build()
    P, G, n_phys, n = 256, 8, 16500, 700           # 16500 * 8 * 256 rows of 128 bytes: 4.3 GB
    k, v = (torch.empty(n_phys, G, P, D, dtype=torch.uint8, device="cuda") for _ in "kv")
    ke, ve = (torch.empty(n_phys, G, P, dtype=torch.uint8, device="cuda") for _ in "kv")
    c = Paged([n], G, 4, P, True, seed=92)
    for j in range(3):
        c.pt[0, j] = n_phys - 1 - j
    c.k, c.v, c.k_exp, c.v_exp, c.n_phys = k, v, ke, ve, n_phys
    c.d.n_phys_pages = n_phys
    new = [torch.randn(1, n, G, D, device="cuda").bfloat16() for _ in "kv"]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    hhr.hhr_append_kv8(c.d, *new, zero, c.seq_len, c.pt, k, v, ke, ve)
    back = [torch.empty(1, n, G, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    hhr.hhr_read_kv8(c.d, k, v, ke, ve, c.pt, zero, c.seq_len, *back)
    q = c.queries(1)
    out, lse = dense(c, q)
    blocks = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda").expand(1, 1, G, 3).contiguous()
    count = torch.full((1, 1, G), 3, dtype=torch.int32, device="cuda")
    out2, lse2 = sparse(c, q[:, None], blocks, count, None)
    status_ok()
    pos = torch.arange(n, device="cuda")
    for name, x, y in zip("kv", new, back):
        rows = torch.stack([c.rows(name, 0, g, pos) for g in range(G)], 1)
        assert torch.equal(y[0].double(), rows)
        ref, exp = quantise_ref(x[0])
        assert torch.equal(rows.cpu(), values_of(ref, exp))
    check_dense(c, q, out, lse)
    check_dense(c, q, out2[:, 0], lse2[:, 0])


def test_cache_rows_past_2_to_31_bytes():
    """Pages whose byte offsets pass 32 bits (a 9 GB pool), the sequence lying at its end."""
    build.build()
    P, G, n_phys = 256, 8, 8200                    # 8200 * 8 * 256 rows of 256 bytes: 4.3 GB
    k = torch.empty(n_phys, G, P, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Paged([700], G, 4, P, False, seed=91)
    for j in range(3):
        src = int(c.pt[0, j])
        k[n_phys - 1 - j], v[n_phys - 1 - j] = c.k[src], c.v[src]
        c.pt[0, j] = n_phys - 1 - j
    c.k, c.v, c.n_phys = k, v, n_phys
    c.d.n_phys_pages = n_phys
    q = c.queries(1)
    out, lse = dense(c, q)
    status_ok()
    check_dense(c, q, out, lse)


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("lens,G,gs,P,T,m,causal", [
    ([40000], 1, 3, 64, 1, 300, False),
    ([30000, 25000], 2, 5, 128, 1, 400, False),
    ([20000], 1, 8, 32, 3, 1000, True),
    ([16000, 300], 2, 4, 16, 2, 1024, True),
    ([9000], 1, 6, 17, 2, 600, False),
    ([12000, 0, 12000], 1, 1, 100, 1, 90, False),
])
def test_long_lists_of_few_rows(lens, G, gs, P, T, m, causal, kv8, per_head):
    """Lists of more than 8192 keys whose rows do not fill the GPU: every row is split evenly over many
    CTAs by its capacity, whatever its count (the whole list, none, one block, a third)."""
    build.build()
    c = Paged(lens, G, gs, P, kv8, seed=131 + P)
    c.d.select_per_head = int(per_head)
    rows = G * gs if per_head else G
    q = c.queries(len(lens), T)
    q_pos = (torch.linspace(max(lens) // 3, max(lens) + 3, T, device="cuda").int().expand(len(lens), T)
             .contiguous() if causal else None)
    gen = torch.Generator(device="cuda").manual_seed(7 * P + T)
    pages = torch.tensor([max(1, -(-n // P)) for n in lens], device="cuda")
    blocks = (torch.rand(len(lens), T, rows, m, generator=gen, device="cuda") *
              pages[:, None, None, None]).int()
    full = [m, 0, 1, m // 3, m]
    count = torch.tensor([full[i % 5] if lens[i // (T * rows)] else 0 for i in range(len(lens) * T * rows)],
                         dtype=torch.int32, device="cuda").reshape(len(lens), T, rows)
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = sparse(c, q, blocks, count, q_pos, dtype)
        status_ok()
        check_sparse(c, q, blocks, count, q_pos, out, lse)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("B,n", [(1, 517), (1, 8000), (1, 131072), (450, 16384)])
@pytest.mark.parametrize("gs", [4, 8])
def test_outputs_are_as_exact_as_fp32_sums(gs, B, n, kv8):
    """The error over all outputs, relative to their size, where errors are independent of one another.
    A weight is off by at most 2^-22 by each of its logit (of size 4), exp2 and its operand parts, by
    2^-22 or less rms in all; over the 190 or more keys that carry a row of 517 an output of 0.25 and
    values of size 1 makes 0.3 of that; a step's and the running fp32 sums add about 2^-24 each. So 2^-22
    is twice what is to be expected. Weights in two bf16 parts (2^-18 each), or sums kept in the matrix
    units' truncating accumulator (a bias that grows with the steps of a warp: 512 where the 450
    sequences, which share their pages, leave every CTA a whole row), are over it."""
    build.build()
    c = Paged([n], 1, gs, 32, kv8, seed=97)
    c.d.batch = B
    c.pt, c.seq_len = c.pt.expand(B, -1).contiguous(), c.seq_len.expand(B).contiguous()
    q = c.queries(B)
    out, lse = dense(c, q)
    status_ok()
    pos = torch.arange(n, device="cuda")
    k, v = c.rows("k", 0, 0, pos), c.rows("v", 0, 0, pos)
    err = size = 0.0
    for b in range(0, B, 60):
        s = SCALE * (q[b].double() @ k.T)
        ref = torch.softmax(s, -1) @ v
        err += float((out[b].double() - ref).square().sum())
        size += float(ref.square().sum())
        assert float((lse[b].double() - torch.logsumexp(s, -1)).abs().max()) < 1e-5
    err = math.sqrt(err / size)
    print(f"relative error {err:.2e}")
    assert err < 2.0 ** -22, err
