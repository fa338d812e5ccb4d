"""The 8-bit cache on the GPU: rows quantised as they are appended, page means, and reading back,
against the format's definition."""
import math

import pytest
import torch

from hash_hierarchical_top_b200 import build, hhr
from page_helpers import D, Paged, quantise_ref, status_ok, values_of

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def new_rows(B, n, G, seed, fused=0):
    """K and V rows [B, n, G, D]: both apart, or slices of a row that also holds `fused` heads."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, n, fused + 2 * G, D, generator=gen, device="cuda")
    # Rows of very different sizes, some channels zero.
    x *= torch.exp2(torch.randint(-40, 40, x.shape[:-1], generator=gen, device="cuda").float())[..., None]
    x[torch.rand(x.shape, generator=gen, device="cuda") < 0.05] = 0
    x = x.bfloat16()
    k, v = x[:, :, fused:fused + G], x[:, :, fused + G:]
    return (k, v) if fused else (k.contiguous(), v.contiguous())


@pytest.mark.parametrize("G,P,start,n_new,fused,mean", [
    (1, 1, [0], [1], 0, True),
    (8, 32, [31, 32, 0], [1, 1, 1], 32, True),            # one token a sequence, slices of Q|K|V
    (2, 5, [0, 3, 17], [23, 0, 9], 0, True),              # pages that end inside the append
    (3, 17, [16, 200], [40, 1], 3, False),
    (1, 256, [255], [300], 0, True),
    (8, 16, [0, 5, 100, 7], [130, 64, 1, 128], 8, True),
    (4, 100, [99, 1], [2, 250], 0, False),
])
def test_append_quantises_and_touches_nothing_else(G, P, start, n_new, fused, mean):
    build.build()
    B = len(start)
    c = Paged([s + n for s, n in zip(start, n_new)], G, 2, P, True, seed=G * 100 + P)
    before = [x.clone() for x in (c.k, c.v, c.k_exp, c.v_exp)]
    means = torch.full((c.n_phys, G, D), 7.0, device="cuda") if mean else None
    k_new, v_new = new_rows(B, max(n_new), G, 3, fused)
    hhr.hhr_append_kv8(c.d, k_new, v_new, i32(start), i32(n_new), c.pt, c.k, c.v, c.k_exp,
                       c.v_exp, means)
    status_ok()
    want = [x.clone() for x in before]
    for b in range(B):
        pos = torch.arange(start[b], start[b] + n_new[b], device="cuda")
        phys, slot = c.pt[b, pos // P].long(), pos % P
        for x, src in ((0, k_new), (1, v_new)):
            q, e = quantise_ref(src[b, :n_new[b]])
            want[x][phys, :, slot] = q.cuda()
            want[x + 2][phys, :, slot] = e.cuda()
    for got, ref, name in zip((c.k, c.v, c.k_exp, c.v_exp), want, ("k", "v", "k_exp", "v_exp")):
        assert torch.equal(got, ref), name
    if not mean:
        return
    touched = torch.zeros(c.n_phys, dtype=torch.bool, device="cuda")
    for b in range(B):
        for lp in range(start[b] // P, -(-(start[b] + n_new[b]) // P) if n_new[b] else 0):
            phys = int(c.pt[b, lp])
            touched[phys] = True
            m = min(P, start[b] + n_new[b] - lp * P)
            x = values_of(c.k[phys, :, :m], c.k_exp[phys, :, :m])
            ref, mag = x.mean(1), x.abs().mean(1)
            # At most P + 16 roundings of fp32 sums, and the division.
            assert ((means[phys].double() - ref).abs() <= (P + 18) * 2.0 ** -24 * mag).all()
    assert (means[~touched] == 7.0).all()


def test_every_bf16_rounds_as_the_format_says():
    """Every finite bf16 magnitude and sign as the second channel of a row whose first one fixes
    the exponent: ties to even, subnormals, zeros of both signs."""
    build.build()
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = bits[torch.isfinite(bits.float())]
    for top in (448.0, 1.0, 2.0 ** -100, 3.0e38, 0.0):
        x = bits[bits.float().abs() <= top] if top else bits[bits == 0]
        n = -(-len(x) // 127)
        rows = torch.zeros(n, D, dtype=torch.bfloat16)
        flat = torch.zeros(n * 127, dtype=torch.bfloat16)
        flat[:len(x)] = x
        rows[:, 1:] = flat.reshape(n, 127)
        rows[:, 0] = top
        rows = rows.reshape(1, n, 1, D).cuda()
        c = Paged([n], 1, 1, 64, True)
        hhr.hhr_append_kv8(c.d, rows, rows, i32([0]), i32([n]), c.pt, c.k, c.v, c.k_exp, c.v_exp)
        status_ok()
        q, e = quantise_ref(rows[0, :, 0])
        pos = torch.arange(n, device="cuda")
        at = (c.pt[0, pos // 64].long(), 0, pos % 64)
        assert torch.equal(c.k_exp[at].cpu(), e)
        assert torch.equal(c.k[at].cpu(), q)
        assert torch.equal(c.v[at].cpu(), q)


def test_infinities_and_nans_stay_in_their_row():
    build.build()
    x = torch.randn(1, 5, 1, D, device="cuda").bfloat16()
    x[0, 1, 0, 3] = math.inf
    x[0, 2, 0, 4] = -math.inf
    x[0, 3, 0, 5] = math.nan
    x[0, 4] = math.nan
    c = Paged([5], 1, 1, 8, True)
    hhr.hhr_append_kv8(c.d, x, x, i32([0]), i32([5]), c.pt, c.k, c.v, c.k_exp, c.v_exp)
    status_ok()
    phys = int(c.pt[0, 0])
    got = values_of(c.k[phys, 0, :5], c.k_exp[phys, 0, :5])
    assert c.k_exp[phys, 0, :5].tolist()[1:3] == [246, 246]
    assert got[1, 3] == 448 * 2.0 ** 119 and got[2, 4] == -448 * 2.0 ** 119
    assert torch.isnan(got[3, 5]) and torch.isfinite(got[3, :5]).all()
    q, e = quantise_ref(x[0, 3, 0])
    keep = torch.arange(D) != 5
    assert torch.equal(c.k[phys, 0, 3].cpu()[keep], q[keep]) and c.k_exp[phys, 0, 3] == e
    assert torch.isnan(got[4]).all() and torch.isfinite(got[0]).all()


def test_append_then_read_back():
    """A ragged append read back whole and in part is the quantised rows, exactly; the rows of
    the outputs past each count keep what they held."""
    build.build()
    G, P, lens = 3, 12, [50, 1, 0, 77]
    c = Paged(lens, G, 1, P, True, seed=5)
    k_new, v_new = new_rows(4, 77, G, 9, fused=2)
    zero, n = i32([0] * 4), i32(lens)
    hhr.hhr_append_kv8(c.d, k_new, v_new, zero, n, c.pt, c.k, c.v, c.k_exp, c.v_exp)
    for start, count in (([0] * 4, lens), ([7, 0, 0, 70], [43, 1, 0, 7]), ([3, 0, 0, 5], [1, 0, 0, 30])):
        k_out = torch.full((4, max(count), G, D), 3.0, dtype=torch.bfloat16, device="cuda")
        v_out = k_out.clone()
        hhr.hhr_read_kv8(c.d, c.k, c.v, c.k_exp, c.v_exp, c.pt, i32(start), i32(count), k_out, v_out)
        status_ok()
        for got, src in ((k_out, k_new), (v_out, v_new)):
            for b in range(4):
                q, e = quantise_ref(src[b, start[b]:start[b] + count[b]])
                ref = values_of(q, e)
                assert torch.equal(got[b, :count[b]].cpu().double(), ref)
                assert (got[b, count[b]:] == 3.0).all()


def test_read_gives_every_value_exactly():
    """All 256 bytes under all exponents that the append writes."""
    build.build()
    exps = torch.arange(10, 247, dtype=torch.uint8, device="cuda")
    n = 2 * len(exps)
    c = Paged([n], 1, 1, 32, True)
    pos = torch.arange(n, device="cuda")
    at = (c.pt[0, pos // 32].long(), 0, pos % 32)
    byte = torch.arange(256, device="cuda").reshape(2, D).to(torch.uint8)
    for x, e in ((c.k, c.k_exp), (c.v, c.v_exp)):
        x[at] = byte.repeat(len(exps), 1)
        e[at] = exps.repeat_interleave(2)
    out = [torch.empty(1, n, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    hhr.hhr_read_kv8(c.d, c.k, c.v, c.k_exp, c.v_exp, c.pt, i32([0]), i32([n]), *out)
    status_ok()
    ref = values_of(byte.repeat(len(exps), 1), exps.repeat_interleave(2))
    for got in out:
        g = got[0, :, 0].double()
        assert torch.equal(torch.isnan(g), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(ref))


def test_bad_pages_and_clipped_counts_are_flagged():
    build.build()
    c = Paged([64, 64], 2, 1, 16, True, seed=2)
    k_new, v_new = new_rows(2, 40, 2, 4)
    c.pt[0, 2] = -1
    c.pt[1, 3] = c.n_phys
    before = [x.clone() for x in (c.k, c.v, c.k_exp, c.v_exp)]
    hhr.hhr_append_kv8(c.d, k_new, v_new, i32([24, 60]), i32([40, 4]), c.pt, c.k, c.v, c.k_exp, c.v_exp)
    torch.cuda.synchronize()
    assert hhr.hhr_read_device_status() == (hhr.HHR_ERR_DEVICE_STATUS, 1)
    pages = c.pt[0, [1, 3]].long()                       # positions 24..31 and 48..63
    untouched = torch.ones(c.n_phys, dtype=torch.bool, device="cuda")
    untouched[pages] = False
    for x, y in zip((c.k, c.v, c.k_exp, c.v_exp), before):
        assert torch.equal(x[untouched], y[untouched])
    assert not torch.equal(c.k[pages[1]], before[0][pages[1]])
    # Counts beyond the rows that are there.
    hhr.hhr_append_kv8(c.d, k_new[:, :4].contiguous(), v_new[:, :4].contiguous(), i32([0, 0]),
                       i32([5, 1]), c.pt, c.k, c.v, c.k_exp, c.v_exp)
    torch.cuda.synchronize()
    assert hhr.hhr_read_device_status() == (hhr.HHR_ERR_DEVICE_STATUS, 4)
    out = [torch.zeros(2, 8, 2, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    hhr.hhr_read_kv8(c.d, c.k, c.v, c.k_exp, c.v_exp, c.pt, i32([30, -2]), i32([9, 2]), *out)
    torch.cuda.synchronize()
    st, bits = hhr.hhr_read_device_status()
    assert (st, bits) == (hhr.HHR_ERR_DEVICE_STATUS, 1 | 2 | 4)
    assert (out[0][0, 2:] == 0).all() and (out[0][1] == 0).all() and (out[0][0, :2] != 0).any()
