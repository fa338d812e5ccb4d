"""The caches and steps together, as a decode loop uses them: a prompt written, then tokens appended
and attended to, dense and block-sparse, in bf16 and 8 bits, beside the hash path on the same cache."""
import math

import pytest
import torch

import hhr_synth as S
from hash_hierarchical_top_b200 import BlockStep, DecodeStep, DenseStep, KV8Cache, LayerCache, build, hhr
from page_helpers import D, check_rows, status_ok, values_of
from parity_helpers import dims_of

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows_of(cache, pt, b, g, pos, P):
    """float64 rows of a KV8Cache: K and V of sequence b, KV head g at pos."""
    phys, slot = pt[b, pos // P].long(), pos % P
    return [values_of(x.view(torch.uint8)[phys, g, slot], e[phys, g, slot])
            for x, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp))]


def test_decode_loop_over_an_8bit_cache():
    """Two layers of one small model: layer 0 dense, layer 1 block-sparse. Every token is written
    (layer 0 by the attention call, layer 1 by the append) and attended to; the dense step is
    captured once and replayed, as a serving loop does."""
    build.build()
    B, G, gs, P, maxp, m = 2, 2, 4, 16, 20, 5
    lens = [100, 33]
    d = hhr.make_dims(B, G * gs, G, P, maxp, B * maxp)
    gen = torch.Generator(device="cuda").manual_seed(3)
    bf = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    pt = torch.randperm(B * maxp, generator=gen, device="cuda").int().reshape(B, maxp)
    caches = [KV8Cache(d, "cuda"), KV8Cache(d, "cuda", block_means=True)]
    dense = DenseStep(d, "cuda", torch.bfloat16)
    block = BlockStep(d, 1, m, "cuda", sink_pages=1, local_pages=1)
    prompt = [bf(B, max(lens), 2 * G, D) for _ in caches]
    for c, x in zip(caches, prompt):
        c.append(x[:, :, :G], x[:, :, G:], i32([0, 0]), i32(lens), pt)
    q, kn, vn = bf(B, G * gs, D), bf(B, G, D), bf(B, G, D)
    seq_len, one = i32(lens), i32([1, 1])
    seq_len += 1
    dense.attend(q, caches[0], pt, seq_len, kn, vn)          # outside a capture first
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dense.attend(q, caches[0], pt, seq_len, kn, vn)
    for step in range(20):
        n = [x + 1 + step for x in lens]
        seq_len.copy_(i32(n))
        q.copy_(bf(B, G * gs, D)); kn.copy_(bf(B, G, D)); vn.copy_(bf(B, G, D))
        graph.replay()
        caches[1].append(kn, vn, seq_len - 1, one, pt)
        out = block.step(q[:, None], caches[1], pt, seq_len)
        status_ok()
        for b in range(B):
            for g in range(G):
                h = slice(g * gs, (g + 1) * gs)
                pos = torch.arange(n[b], device="cuda")
                k, v = rows_of(caches[0], pt, b, g, pos, P)
                check_rows(dense.out[b, h], dense.lse[b, h], q[b, h], k, v, SCALE, f"dense {step}")
                mine = block.blocks[b, 0, g, :int(block.count[b, 0, g])].tolist()
                pages = -(-n[b] // P)
                assert len(mine) == min(m, pages) and 0 in mine and pages - 1 in mine
                k, v = rows_of(caches[1], pt, b, g, pos, P)
                means = torch.stack([k[p * P:(p + 1) * P].mean(0) for p in range(pages)])
                s = means @ q[b, h].double().sum(0)
                left = [p for p in range(pages) if p not in mine]
                if left:   # fp32 means: scores may differ by their rounding
                    free = [p for p in mine if p not in (0, pages - 1)]
                    assert s[free].min() >= s[left].max() - 1e-4
                at = torch.cat([torch.arange(p * P, min(n[b], (p + 1) * P)) for p in mine]).cuda()
                check_rows(out[b, 0, h], block.lse[b, 0, h], q[b, h], k[at], v[at], SCALE, f"block {step}")
    k_out, v_out = (torch.zeros(B, max(lens) + 20, G, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    caches[0].read(i32([0, 0]), seq_len, pt, k_out, v_out)
    status_ok()
    for b in range(B):
        for g in range(G):
            k, v = rows_of(caches[0], pt, b, g, torch.arange(int(seq_len[b]), device="cuda"), P)
            assert torch.equal(k_out[b, :len(k), g].double(), k)
            assert torch.equal(v_out[b, :len(v), g].double(), v)


def test_steps_beside_the_hash_path_on_one_bf16_cache():
    """The hash step, dense attention and block attention on the same cache and page table: the
    dense step is the hash step with every key selected; block attention takes the pages that the
    hash path's bounds kept (its trace) and those of the block means that the encoder writes."""
    build.build()
    wl = S.scaled(S.WORKLOADS["llama8b_32k"], batch=2, seq_lens=(3000, 1700), top_k=3200, m_pages=12,
                  keep_div=0)
    inp = S.make_inputs(wl, device="cuda")
    d = dims_of(wl, inp)
    P, G, gs = wl.page_size, wl.n_kv_heads, wl.n_q_heads // wl.n_kv_heads
    cache = LayerCache(d, "cuda", block_means=True)
    zero = i32([0, 0])
    hashed = DecodeStep(d, hhr.HHR_MODE_HASH, wl.m_pages, 0, wl.top_k, "cuda")
    # The per-page encoder writes the block means too.
    hhr.hhr_encode_keys(d, inp["k_cache"], inp["page_table"], zero, inp["seq_len"], 3000, inp["R"],
                        inp["W"], cache.page_minmax, cache.codes, cache.block_mean)
    kept = torch.empty(2, G, hashed.m_max, dtype=torch.int32, device="cuda")
    kept_count = torch.empty(2, G, dtype=torch.int32, device="cuda")
    hashed.select(inp["q"], inp["seq_len"], inp["page_table"], cache, R=inp["R"], W=inp["W"],
                  trace=hhr.make_trace(kept=kept, kept_count=kept_count))
    pair = (inp["k_cache"], inp["v_cache"])

    def logical(x, b, g, pos):
        return x[inp["page_table"][b, pos // P].long(), g, pos % P].double()

    def check(out, lse, blocks, count, what):
        for b, n in enumerate(wl.seq_lens):
            for g in range(G):
                pos = (blocks[b, g, :int(count[b, g])].long()[:, None] * P +
                       torch.arange(P, device="cuda")).reshape(-1)
                pos = pos[pos < n]
                h = slice(g * gs, (g + 1) * gs)
                check_rows(out[b, h], lse[b, h], inp["q"][b, h], logical(pair[0], b, g, pos),
                           logical(pair[1], b, g, pos), SCALE, what)

    block = BlockStep(d, 1, wl.m_pages, "cuda")
    block.blocks.copy_(kept[:, None])
    block.count.copy_(kept_count[:, None])
    block.attend(inp["q"][:, None], pair, inp["page_table"], inp["seq_len"])
    status_ok()
    check(block.out[:, 0], block.lse[:, 0], kept, kept_count, "kept pages")
    block.step(inp["q"][:, None], pair, inp["page_table"], inp["seq_len"], cache.block_mean)
    status_ok()
    assert (block.count == wl.m_pages).all()
    check(block.out[:, 0], block.lse[:, 0], block.blocks[:, 0], block.count[:, 0], "mean blocks")
    dense = DenseStep(d, "cuda")
    dense.attend(inp["q"], pair, inp["page_table"], inp["seq_len"])
    pages = inp["page_table"].shape[1]
    every = torch.arange(pages, dtype=torch.int32, device="cuda").expand(2, G, pages)
    check(dense.out, dense.lse, every, torch.full((2, G), pages), "dense")
    idx = torch.arange(3200, dtype=torch.int32, device="cuda").expand(2, G, 3200).contiguous()
    hashed.idx.copy_(idx)
    hashed.count.copy_(inp["seq_len"].view(2, 1).expand(2, G))
    hashed.attend(inp["q"], *pair, inp["page_table"], inp["seq_len"])
    status_ok()
    # Both within 2e-3 of the formula relative to the row's largest channel (the token-list
    # attention's stated tolerance), so within twice that of one another.
    top = dense.out.abs().amax(-1, keepdim=True)
    assert ((dense.out - hashed.out).abs() <= 4e-3 * top).all()


def test_unsupported_sizes_are_refused():
    d = hhr.make_dims(1, 8, 2, 16, 4, 4, head_dim=64)
    for make in (lambda: DenseStep(d, "cuda"), lambda: BlockStep(d, 1, 2, "cuda"),
                 lambda: BlockStep(hhr.make_dims(1, 8, 2, 16, 4, 4), 0, 2, "cuda"),
                 lambda: BlockStep(hhr.make_dims(1, 8, 2, 16, 4, 4), 1, 0, "cuda")):
        with pytest.raises(ValueError):
            make()


@pytest.mark.parametrize("own_stream", [False, True])
def test_a_dense_step_keeps_the_block_means(own_stream):
    """Tokens appended by dense steps to a cache with block means: the means are those of the rows, so
    that a block-sparse step can follow; rows and outputs are those of a cache without means."""
    build.build()
    B, G, gs, P, maxp = 3, 2, 4, 8, 9
    lens = [13, 0, 40]
    d = hhr.make_dims(B, G * gs, G, P, maxp, B * maxp)
    gen = torch.Generator(device="cuda").manual_seed(23)
    bf = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    pt = torch.randperm(B * maxp, generator=gen, device="cuda").int().reshape(B, maxp)
    with_means, plain = KV8Cache(d, "cuda", block_means=True), KV8Cache(d, "cuda")
    prompt = bf(B, max(lens), 2 * G, D)
    for c in (with_means, plain):
        c.append(prompt[:, :, :G], prompt[:, :, G:], i32([0] * B), i32(lens), pt)
    steps = DenseStep(d, "cuda"), DenseStep(d, "cuda")
    stream = torch.cuda.Stream() if own_stream else None
    block = BlockStep(d, 1, 3, "cuda")
    for step in range(1, 19):
        # Sequence 1 stays empty for a while: nothing of it is written.
        n = [lens[0] + step, max(0, step - 5), lens[2] + step]
        seq_len, q, kn, vn = i32(n), bf(B, G * gs, D), bf(B, G, D), bf(B, G, D)
        torch.cuda.synchronize()
        a = steps[0].attend(q, with_means, pt, seq_len, kn, vn, stream=stream)
        torch.cuda.synchronize()
        b = steps[1].attend(q, plain, pt, seq_len, kn, vn)
        status_ok()
        assert torch.equal(a, b) and torch.equal(steps[0].lse, steps[1].lse)
        for x, y in ((with_means.k, plain.k), (with_means.v, plain.v)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert torch.equal(with_means.k_exp, plain.k_exp) and torch.equal(with_means.v_exp, plain.v_exp)
    for b in range(B):
        for g in range(G):
            k, _ = rows_of(with_means, pt, b, g, torch.arange(n[b], device="cuda"), P)
            for p in range(-(-n[b] // P)):
                x = k[p * P:(p + 1) * P]
                err = (with_means.block_mean[int(pt[b, p]), g].double() - x.mean(0)).abs()
                # At most P + 16 roundings of fp32 sums, and the division.
                assert (err <= (P + 18) * 2.0 ** -24 * x.abs().mean(0)).all(), (b, g, p)
    block.step(q[:, None], with_means, pt, seq_len)
    status_ok()
    assert block.count[:, 0, 0].tolist() == [min(3, -(-x // P)) for x in n]


def test_a_captured_dense_step_keeps_the_block_means():
    build.build()
    B, G, P, maxp = 2, 1, 4, 6
    d = hhr.make_dims(B, 2, G, P, maxp, B * maxp)
    pt = torch.arange(B * maxp, dtype=torch.int32, device="cuda").reshape(B, maxp)
    cache, step = KV8Cache(d, "cuda", block_means=True), DenseStep(d, "cuda")
    q, kn, vn = (torch.randn(B, h, D, device="cuda").bfloat16() for h in (2, 1, 1))
    seq_len = i32([0, 0])
    step.attend(q, cache, pt, seq_len, kn, vn)               # outside a capture first: writes nothing
    torch.cuda.synchronize()
    assert not cache.k_exp.any() and not cache.block_mean.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.attend(q, cache, pt, seq_len, kn, vn)
    for n in range(1, 11):
        seq_len.copy_(i32([n, max(0, n - 4)]))
        kn.normal_()
        graph.replay()
        status_ok()
    for b, n in ((0, 10), (1, 6)):
        k, _ = rows_of(cache, pt, b, 0, torch.arange(n, device="cuda"), P)
        for p in range(-(-n // P)):
            x = k[p * P:(p + 1) * P]
            err = (cache.block_mean[int(pt[b, p]), 0].double() - x.mean(0)).abs()
            assert (err <= (P + 18) * 2.0 ** -24 * x.abs().mean(0)).all()


def test_a_refused_dense_step_writes_nothing_and_buffers_may_be_larger():
    """The checks come before the append that keeps the means; new rows and lengths in buffers of a larger
    batch, and new rows as [B, G d], are taken as without means."""
    build.build()
    B, G, P, maxp = 2, 2, 4, 6
    d = hhr.make_dims(B, 4, G, P, maxp, B * maxp)
    pt = torch.arange(B * maxp, dtype=torch.int32, device="cuda").reshape(B, maxp)
    cache, step = KV8Cache(d, "cuda", block_means=True), DenseStep(d, "cuda")
    q, kn, vn = (torch.randn(4, h, D, device="cuda").bfloat16() for h in (4, 2, 2))
    n = i32([5, 3, 9, 9])
    for bad in (dict(q=q.float()), dict(seq_len=n.long()), dict(v_new=None), dict(k_new=kn.cpu())):
        a = dict(q=q, cache=cache, page_table=pt, seq_len=n, k_new=kn, v_new=vn)
        with pytest.raises((TypeError, ValueError, hhr.HHRError)):
            step.attend(**{**a, **bad})
    status_ok()
    assert not cache.k_exp.any() and not cache.v_exp.any() and not cache.block_mean.any()
    step.attend(q, cache, pt, n, kn, vn)
    means = cache.block_mean.clone()
    step.attend(q, cache, pt, n, kn.reshape(4, -1), vn.reshape(4, -1))
    status_ok()
    assert torch.equal(cache.block_mean, means) and means.any() and int((cache.k_exp != 0).sum()) == B * G
    assert step.newest.start.tolist() == [4, 2]


@pytest.mark.parametrize("with_new_rows", [False, True])
def test_a_fused_step_keeps_the_block_means(with_new_rows):
    """Tokens appended by fused hash steps to a cache with block means: the means are the encoder's, bit for
    bit, and the hash metadata and outputs those of a cache without means."""
    build.build()
    wl = S.scaled(S.WORKLOADS["llama8b_32k"], batch=2, seq_lens=(300, 170), top_k=64, m_pages=4, keep_div=0)
    inp = S.make_inputs(wl, device="cuda")
    d = dims_of(wl, inp)
    zero, P = i32([0, 0]), wl.page_size
    caches = [LayerCache(d, "cuda", block_means=True), LayerCache(d, "cuda"), LayerCache(d, "cuda", block_means=True)]
    steps = [DecodeStep(d, hhr.HHR_MODE_HASH, wl.m_pages, 0, wl.top_k, "cuda") for _ in range(2)]
    kv = [(inp["k_cache"].clone(), inp["v_cache"].clone()) for _ in range(2)]
    first = [x - 40 for x in wl.seq_lens]
    for c in caches[:2]:
        hhr.hhr_encode_keys(d, inp["k_cache"], inp["page_table"], zero, i32(first), max(first), inp["R"], inp["W"],
                            c.page_minmax, c.codes, c.block_mean)
    gen = torch.Generator(device="cuda").manual_seed(29)
    for t in range(1, 41):
        n = i32([x + t for x in first])
        q = torch.randn(2, wl.n_q_heads, D, generator=gen, device="cuda").bfloat16()
        new = [torch.randn(2, wl.n_kv_heads, D, generator=gen, device="cuda").bfloat16() if with_new_rows else None
               for _ in "kv"]
        for step, c, (k, v) in zip(steps, caches, kv):
            step.fused_step(q, k, v, inp["page_table"], n, inp["R"], inp["W"], c, k_new=new[0], v_new=new[1])
        status_ok()
        assert torch.equal(steps[0].out, steps[1].out) and torch.equal(steps[0].idx, steps[1].idx)
    assert torch.equal(caches[0].codes, caches[1].codes)
    assert torch.equal(caches[0].page_minmax, caches[1].page_minmax)
    hhr.hhr_encode_keys(d, kv[0][0], inp["page_table"], zero, n, max(wl.seq_lens), None, None, None, None,
                        caches[2].block_mean)
    status_ok()
    assert torch.equal(caches[0].block_mean, caches[2].block_mean) and caches[0].block_mean.any()
