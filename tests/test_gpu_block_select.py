"""Block selection on the GPU against the definition: 64-bit scores rounded to fp32 once, the m
largest, ties to the lower block. Sets are compared exactly: a 64-bit sum in another order is off
by 2^-45 of its terms, which moves an fp32 rounding about once in a million scores, and a set only
where that score lies at the cut."""
import math

import pytest
import torch

from hash_hierarchical_top_b200 import build, hhr
from page_helpers import D, Paged, check_rows, status_ok

pytestmark = pytest.mark.gpu


def reference(q, means, pt, lens, q_pos, P, rows, m, sink=0, local=0):
    B, T, Hq, _ = q.shape
    G = means.shape[1]
    gs = Hq // rows
    blocks = torch.full((B, T, rows, m), -1, dtype=torch.int32)
    count = torch.zeros(B, T, rows, dtype=torch.int32)
    q, means = q.double().cpu(), means.double().cpu()
    for b in range(B):
        for t in range(T):
            limit = lens[b] if q_pos is None else min(lens[b], int(q_pos[b, t]) + 1)
            n = max(0, -(-limit // P))
            for r in range(rows):
                mean = means[pt[b, :n].long().cpu(), r * G // rows]
                s = (mean @ q[b, t, r * gs:(r + 1) * gs].sum(0)).float()
                s[torch.isnan(s)] = -math.inf
                forced = torch.zeros(n, dtype=torch.bool)
                forced[:sink] = True
                forced[max(0, n - local):] = True
                s[forced] = math.inf
                order = s.sort(descending=True, stable=True).indices
                k = min(m, int((s > -math.inf).sum()))
                blocks[b, t, r, :k] = order[:k].sort().values.int()
                count[b, t, r] = k
    return blocks, count


def select(d, q, seq_len, q_pos, pt, means, m, opts=None):
    rows, m_max = hhr.sel_rows(d), hhr.hhr_kept_max(d, m, 0)
    blocks = torch.full((d.batch, q.shape[1], rows, m_max), -7, dtype=torch.int32, device="cuda")
    count = torch.full((d.batch, q.shape[1], rows), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((hhr.hhr_block_select_workspace_bytes(d, q.shape[1]),), 0xff, dtype=torch.uint8,
                    device="cuda")
    hhr.hhr_block_select(d, q, seq_len, q_pos, pt, means, m, blocks, count, ws, opts=opts)
    return blocks, count


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("lens,G,gs,P,T,m,sink,local,causal", [
    ([1], 1, 1, 1, 1, 1, 0, 0, False),
    ([0, 5, 700], 2, 4, 32, 1, 4, 0, 0, False),
    ([1000, 3000, 37], 8, 4, 16, 3, 20, 1, 2, True),
    ([9000], 1, 8, 5, 9, 256, 0, 1, True),
    ([40000, 100], 2, 3, 32, 2, 64, 2, 0, False),
    ([8192], 4, 4, 128, 64, 16, 0, 1, True),
    ([20000], 1, 5, 1, 1, 300, 1, 1, False),
    ([640], 3, 7, 256, 4, 3, 1, 1, True),
])
def test_sets_match_the_definition(lens, G, gs, P, T, m, sink, local, causal, per_head):
    build.build()
    gen = torch.Generator(device="cuda").manual_seed(P + T)
    B, pages = len(lens), [-(-n // P) for n in lens]
    maxp, n_phys = max(pages + [m]), sum(pages) + 3
    pt = torch.full((B, maxp), -1, dtype=torch.int32, device="cuda")
    order, at = torch.randperm(n_phys, generator=gen, device="cuda").int(), 0
    for b, n in enumerate(pages):
        pt[b, :n] = order[at:at + n]
        at += n
    d = hhr.make_dims(B, G * gs, G, P, maxp, n_phys, select_per_head=int(per_head))
    means = torch.randn(n_phys, G, D, generator=gen, device="cuda")
    q = torch.randn(B, T, G * gs, D, generator=gen, device="cuda").bfloat16()
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q_pos = (torch.linspace(-1, max(lens) + 3, T, device="cuda").int().expand(B, T).contiguous()
             if causal else None)
    blocks, count = select(d, q, seq_len, q_pos, pt, means, m, hhr.make_opts(sink, local))
    status_ok()
    ref_blocks, ref_count = reference(q, means, pt, lens, q_pos, P, hhr.sel_rows(d), m, sink, local)
    assert torch.equal(count.cpu(), ref_count)
    assert torch.equal(blocks.cpu(), ref_blocks)


def test_ties_zeros_and_non_finite_scores():
    """Equal scores and zeros of both signs go to the lower block, NaN and -inf scores are never
    kept (unless forced), +inf ones are."""
    build.build()
    P, n = 8, 40
    d = hhr.make_dims(1, 2, 1, P, n, n)
    pt = torch.arange(n, dtype=torch.int32, device="cuda").reshape(1, n)
    means = torch.zeros(n, 1, D, device="cuda")
    q = torch.ones(1, 1, 2, D, device="cuda").bfloat16()
    seq_len = torch.tensor([n * P], dtype=torch.int32, device="cuda")

    def ask(m, opts=None):
        blocks, count = select(d, q, seq_len, None, pt, means, m, opts)
        status_ok()
        return blocks[0, 0, 0, :int(count)].tolist()

    assert ask(5) == [0, 1, 2, 3, 4]
    means[0] = -0.0
    means[7] = 1.0
    assert ask(3) == [0, 1, 7]
    means[1, 0, 0] = math.nan
    means[2, 0, 0] = -math.inf
    means[30, 0, 0] = math.inf
    assert ask(4) == [0, 3, 7, 30]
    assert ask(40) == [i for i in range(40) if i not in (1, 2)]
    assert ask(4, hhr.make_opts(2, 1)) == [0, 1, 30, 39]


@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("kind", ["levels", "equal", "huge", "tiny", "mixed", "close"])
def test_many_ties_and_extreme_sizes(kind, T):
    """Scores that crowd at the cut: few distinct means, equal ones, sizes past what fp32 squares
    hold, blocks of very different sizes, and scores that differ in the last bits only."""
    build.build()
    P, n, G, m = 16, 2500, 2, 100
    gen = torch.Generator(device="cuda").manual_seed(7)
    means = torch.randn(n + 1, G, D, generator=gen, device="cuda")
    if kind == "levels":
        means = means[torch.randint(0, 9, (n + 1,), generator=gen, device="cuda")].clone()
    elif kind == "equal":
        means = means[:1].expand(n + 1, G, D).contiguous()
    elif kind == "huge":
        means *= 1e25
    elif kind == "tiny":
        means *= 1e-25
    elif kind == "mixed":
        means *= torch.exp2(torch.randint(-60, 30, (n + 1, 1, 1), generator=gen, device="cuda").float())
    else:
        means = means[:1] * (1 + 1e-6 * torch.randn(n + 1, G, 1, generator=gen, device="cuda"))
    means = means.contiguous()
    d = hhr.make_dims(2, 4, G, P, n, n + 1)
    pt = torch.stack([torch.randperm(n + 1, generator=gen, device="cuda")[:n] for _ in "ab"]).int()
    lens = [n * P, 2000 * P - 3]
    q = torch.randn(2, T, 4, D, generator=gen, device="cuda").bfloat16()
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for opts in (None, hhr.make_opts(3, 2)):
        blocks, count = select(d, q, seq_len, None, pt, means, m, opts)
        status_ok()
        ref = reference(q, means, pt, lens, None, P, G, m, *((3, 2) if opts else (0, 0)))
        assert torch.equal(count.cpu(), ref[1]) and torch.equal(blocks.cpu(), ref[0])


def test_long_rows_and_captured_calls():
    """32768 blocks a sequence (keys past the narrow and the wide choice's registers), and the
    call captured once and replayed on other inputs."""
    build.build()
    P, n, G, m = 4, 32768, 1, 2000
    gen = torch.Generator(device="cuda").manual_seed(9)
    means = torch.randn(n, G, D, generator=gen, device="cuda")
    d = hhr.make_dims(1, 3, G, P, n, n)
    pt = torch.randperm(n, generator=gen, device="cuda").int().reshape(1, n)
    q = torch.randn(1, 1, 3, D, generator=gen, device="cuda").bfloat16()
    seq_len = torch.tensor([n * P], dtype=torch.int32, device="cuda")
    blocks = torch.empty(1, 1, 1, m, dtype=torch.int32, device="cuda")
    count = torch.empty(1, 1, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(hhr.hhr_block_select_workspace_bytes(d, 1), dtype=torch.uint8, device="cuda")
    call = lambda: hhr.hhr_block_select(d, q, seq_len, None, pt, means, m, blocks, count, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for length in (n * P, 7777, 0, 1):
        q.copy_(torch.randn(1, 1, 3, D, generator=gen, device="cuda").bfloat16())
        seq_len.fill_(length)
        graph.replay()
        status_ok()
        ref = reference(q, means, pt, [length], None, P, 1, m)
        assert torch.equal(count.cpu(), ref[1]) and torch.equal(blocks.cpu(), ref[0])


@pytest.mark.parametrize("T", [1, 2])
def test_many_ragged_sequences(T):
    """More sequences than a warp scans at once, empty ones among them."""
    build.build()
    P, G, m = 8, 2, 6
    gen = torch.Generator(device="cuda").manual_seed(11)
    lens = [(53 * i) % 700 if i % 7 else 0 for i in range(90)]
    pages = [-(-n // P) for n in lens]
    maxp, n_phys = max(pages), sum(pages)
    pt = torch.full((90, maxp), -1, dtype=torch.int32, device="cuda")
    order, at = torch.randperm(n_phys, generator=gen, device="cuda").int(), 0
    for b, n in enumerate(pages):
        pt[b, :n] = order[at:at + n]
        at += n
    means = torch.randn(n_phys, G, D, generator=gen, device="cuda")
    d = hhr.make_dims(90, 6, G, P, maxp, n_phys)
    q = torch.randn(90, T, 6, D, generator=gen, device="cuda").bfloat16()
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    blocks, count = select(d, q, seq_len, None, pt, means, m)
    status_ok()
    ref = reference(q, means, pt, lens, None, P, G, m)
    assert torch.equal(count.cpu(), ref[1]) and torch.equal(blocks.cpu(), ref[0])


def test_many_kv_heads():
    """More KV heads than the single-token stream stages."""
    build.build()
    G, P, n = 70, 8, 200
    gen = torch.Generator(device="cuda").manual_seed(10)
    means = torch.randn(n, G, D, generator=gen, device="cuda")
    d = hhr.make_dims(1, 2 * G, G, P, n, n)
    pt = torch.randperm(n, generator=gen, device="cuda").int().reshape(1, n)
    q = torch.randn(1, 1, 2 * G, D, generator=gen, device="cuda").bfloat16()
    lens = [n * P - 3]
    blocks, count = select(d, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), None, pt, means, 17)
    status_ok()
    ref = reference(q, means, pt, lens, None, P, G, 17)
    assert torch.equal(count.cpu(), ref[1]) and torch.equal(blocks.cpu(), ref[0])


def test_blocks_without_a_page_are_flagged_and_not_kept():
    build.build()
    c = Paged([320], 2, 2, 32, False, seed=5)
    means = torch.randn(c.n_phys, 2, D, device="cuda")
    q = c.queries(1, 1)
    c.pt[0, 4] = c.n_phys
    blocks, count = select(c.d, q, c.seq_len, None, c.pt, means, 10)
    torch.cuda.synchronize()
    assert hhr.hhr_read_device_status() == (hhr.HHR_ERR_DEVICE_STATUS, 1)
    assert (count == 9).all() and not (blocks == 4).any()


@pytest.mark.parametrize("T", [1, 5])
def test_append_select_attend(T):
    """A prompt and then tokens appended to an 8-bit cache, their blocks selected by the means
    that the append keeps, and attended to: the chain of calls of a block-sparse layer. Each
    call's inputs are the previous ones' outputs, and each is checked on those."""
    build.build()
    lens, G, gs, P, m = [900, 333], 2, 4, 32, 6
    B = len(lens)
    c = Paged(lens, G, gs, P, True, seed=17)
    means = torch.zeros(c.n_phys, G, D, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(18)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(B, max(lens), G, D, generator=gen, device="cuda").bfloat16() for _ in "kv")
    prompt = [n - T for n in lens]
    hhr.hhr_append_kv8(c.d, k, v, i32([0] * B), i32(prompt), c.pt, c.k, c.v, c.k_exp, c.v_exp, means)
    kt = torch.stack([k[b, n - T:n] for b, n in enumerate(lens)])
    vt = torch.stack([v[b, n - T:n] for b, n in enumerate(lens)])
    hhr.hhr_append_kv8(c.d, kt, vt, i32(prompt), i32([T] * B), c.pt, c.k, c.v, c.k_exp, c.v_exp, means)
    q = c.queries(B, T)
    q_pos = i32([[n - T + t for t in range(T)] for n in lens])
    opts = hhr.make_opts(1, 1)
    blocks, count = select(c.d, q, c.seq_len, q_pos, c.pt, means, m, opts)
    out = torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:-1], device="cuda")
    ws = torch.empty(hhr.hhr_block_attn_workspace_bytes(c.d, T, m), dtype=torch.uint8, device="cuda")
    hhr.hhr_block_attn(c.d, q, c.k, c.v, c.k_exp, c.v_exp, c.pt, c.seq_len, q_pos, blocks, count,
                       1 / math.sqrt(D), out, ws, lse=lse)
    status_ok()
    ref_blocks, ref_count = reference(q, means, c.pt, lens, q_pos, P, G, m, 1, 1)
    assert torch.equal(blocks.cpu(), ref_blocks) and torch.equal(count.cpu(), ref_count)
    for b, n in enumerate(lens):
        for g in range(G):
            whole = c.rows("k", b, g, torch.arange(n, device="cuda"))
            for p in range(-(-n // P)):
                x = whole[p * P:(p + 1) * P]
                err = (means[int(c.pt[b, p]), g].double() - x.mean(0)).abs()
                assert (err <= (P + 18) * 2.0 ** -24 * x.abs().mean(0)).all()
            for t in range(T):
                pos = (blocks[b, t, g, :int(count[b, t, g])].long()[:, None] * P +
                       torch.arange(P, device="cuda")).reshape(-1)
                pos = pos[pos <= n - T + t]
                h = slice(g * gs, (g + 1) * gs)
                check_rows(out[b, t, h], lse[b, t, h], q[b, t, h], c.rows("k", b, g, pos),
                           c.rows("v", b, g, pos), 1 / math.sqrt(D), f"{b} {g} {t}")


@pytest.mark.parametrize("kind", ["ordinary", "huge", "nan"])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("sink,local", [(1, 0), (0, 1), (1, 2), (3, 1), (0, 64)])
def test_every_kept_block_is_forced(sink, local, T, kind):
    """As many blocks kept as are forced, and one more (the best of the rest): with scores that fp32
    holds, and with ones that it does not."""
    build.build()
    P, G, lens = 16, 2, [3000 * 16, 37, 65 * 16 - 1]
    gen = torch.Generator(device="cuda").manual_seed(13)
    pages = [-(-n // P) for n in lens]
    maxp, n_phys = max(pages), sum(pages)
    means = torch.randn(n_phys, G, D, generator=gen, device="cuda")
    if kind == "huge":
        means *= 1e37
    elif kind == "nan":
        means[::7, :, 3] = math.nan
    pt = torch.full((3, maxp), -1, dtype=torch.int32, device="cuda")
    order, at = torch.randperm(n_phys, generator=gen, device="cuda").int(), 0
    for b, n in enumerate(pages):
        pt[b, :n] = order[at:at + n]
        at += n
    d = hhr.make_dims(3, 8, G, P, maxp, n_phys)
    q = torch.randn(3, T, 8, D, generator=gen, device="cuda").bfloat16()
    seq_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for m in (sink + local, sink + local + 1):
        blocks, count = select(d, q, seq_len, None, pt, means, m, hhr.make_opts(sink, local))
        status_ok()
        for b, n in enumerate(pages):
            forced = set(range(min(sink, n))) | set(range(max(0, n - local), n))
            for g in range(G):
                mean = means[pt[b, :n].long(), g].double()
                for t in range(T):
                    s = (mean @ q[b, t, 4 * g:4 * g + 4].double().sum(0)).float().tolist()
                    # (Forced blocks come before any score: huge ones are +inf in fp32.)
                    rest = sorted((-x, p) for p, x in enumerate(s) if x > -math.inf and p not in forced)
                    want = sorted(list(forced) + [p for _, p in rest[:max(0, m - len(forced))]])
                    assert blocks[b, t, g, :int(count[b, t, g])].tolist() == want
                    assert (blocks[b, t, g, len(want):] == -1).all()
