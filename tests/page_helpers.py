"""Inputs and 64-bit references of the 8-bit cache and the page attentions.

The references are written from the definitions in include/hhr.h, in float64, one row at a time.
Tolerances, per output channel, for rows of n keys (all of them worst cases added up):
  * a logit: 128 exact products summed in fp32 by 8 matrix steps, each off by at most 2 units
    of the last place of its partial sums: 2^-19 sum_c |q_c k_c| scale, plus a few roundings of
    the logit itself, 2^-22 |s| (scale, log2 e, exponent, difference to the maximum); ds = the
    largest of these over the row. A weight exp(s - max) is then off by ds, relative, and the
    weights' sum by as much again;
  * a weight as operand parts: 2^-21 (f16: 2^-11 of a remainder of 2^-11; bf16 parts leave less);
  * sums of n weights and n weighted values, 16 or 32 keys a step over at least 8 warps:
    (n / 128 + 64) 2^-22 of the sum of magnitudes (the 64: joins of warps and of splits, exp2);
  so |o - o_ref| <= (2 ds + 2^-21 + (n / 128 + 64) 2^-22) sum_j w_j |v_jc|, plus 2^-8 |o_ref| for
  a bf16 output, and |lse - lse_ref| <= ds + (n / 128 + 64) 2^-22 + 2^-22 |lse_ref|.
"""
from __future__ import annotations

import math

import torch

from hash_hierarchical_top_b200 import hhr

D = 128


def e4m3_values():
    """The values of the 256 e4m3 bytes, from the format: 1 sign, 4 exponent (bias 7), 3
    significand bits; 0x7f and 0xff are NaN."""
    v = []
    for b in range(256):
        s, e, m = -1.0 if b & 128 else 1.0, (b >> 3) & 15, b & 7
        v.append(math.nan if (e, m) == (15, 7) else
                 s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)))
    return torch.tensor(v, dtype=torch.float64)


def quantise_ref(x):
    """(bytes, exponent bytes) of bf16 rows x [..., 128], on the CPU, by the definition."""
    x = x.cpu().double()
    mag = x.abs()
    top = torch.where(torch.isnan(mag), torch.zeros_like(mag), mag).amax(-1)
    e = torch.full(top.shape, 119, dtype=torch.int64)
    for cand in range(118, -118, -1):      # the smallest e with top <= 448 * 2^e
        e = torch.where(top <= 448 * 2.0 ** cand, torch.full_like(e, cand), e)
    y = x * torch.exp2(-e.double())[..., None]
    table = e4m3_values()
    pos = table[:127]                        # 0 .. 448, ascending
    mag = y.abs().clamp(max=448.0)
    hi = torch.searchsorted(pos, torch.nan_to_num(mag).contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = mag - pos[lo], pos[hi] - mag
    near = torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(lo % 2 == 0, lo, hi)))
    byte = near + 128 * torch.signbit(y)
    byte = torch.where(torch.isnan(y), torch.full_like(byte, 127), byte)
    return byte.to(torch.uint8), (e + 127).to(torch.uint8)


def values_of(byte, exp):
    """float64 rows that bytes [..., 128] and exponent bytes [...] stand for."""
    return e4m3_values().to(byte.device)[byte.view(torch.uint8).long()] * \
        torch.exp2(exp.double() - 127)[..., None]


class Paged:
    """A paged cache of B sequences in a permuted pool; slots that hold no key are filled with
    NaNs (and, in 8 bits, with the largest exponent)."""

    def __init__(self, lens, G, gs, P, kv8, seed=0, spare=2, extra_cols=1, scale=1.0):
        dev = "cuda"
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.lens, self.G, self.gs, self.P, self.kv8 = list(lens), G, gs, P, kv8
        B = len(self.lens)
        pages = [-(-n // P) for n in self.lens]
        self.maxp = max(pages + [1]) + extra_cols
        self.n_phys = sum(pages) + spare
        order = torch.randperm(self.n_phys, generator=gen, device=dev)
        self.pt = torch.full((B, self.maxp), -1, dtype=torch.int32, device=dev)
        at = 0
        held = torch.zeros(self.n_phys, P, dtype=torch.bool, device=dev)
        for b, n in enumerate(pages):
            self.pt[b, :n] = order[at:at + n].int()
            at += n
            for j in range(n):
                held[self.pt[b, j].long(), :min(P, self.lens[b] - j * P)] = True
        self.seq_len = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        shape = (self.n_phys, G, P, D)
        k = torch.randn(shape, generator=gen, device=dev) * scale
        k[..., 5::37] *= 5
        v = torch.randn(shape, generator=gen, device=dev) + 0.25
        empty = ~held[:, None, :].expand(self.n_phys, G, P)
        if kv8:
            (kq, kx), (vq, vx) = (quantise_ref(x.bfloat16()) for x in (k, v))
            self.k, self.v = kq.to(dev), vq.to(dev)
            self.k_exp, self.v_exp = kx.to(dev), vx.to(dev)
            for x, e in ((self.k, self.k_exp), (self.v, self.v_exp)):
                x[empty] = 0x7f
                e[empty] = 255
        else:
            self.k, self.v, self.k_exp, self.v_exp = k.bfloat16(), v.bfloat16(), None, None
            self.k[empty] = math.nan
            self.v[empty] = math.nan
        self.gen = gen
        self.d = hhr.make_dims(B, G * gs, G, P, self.maxp, self.n_phys)

    def rows(self, name, b, g, pos):
        """float64 rows of sequence b, KV head g at the positions pos."""
        phys, slot = self.pt[b, pos // self.P].long(), pos % self.P
        x = getattr(self, name)[phys, g, slot]
        if not self.kv8:
            return x.double()
        return values_of(x, getattr(self, name + "_exp")[phys, g, slot])

    def queries(self, *lead):
        return torch.randn(*lead, self.G * self.gs, D, generator=self.gen,
                           device="cuda").bfloat16()


def attend_ref(q, k, v, scale):
    """(o, lse, tolerance of o, tolerance of lse) of q [h, D] over rows k, v [n, D], float64."""
    q, n = q.double(), len(k)
    h = len(q)
    if n == 0:
        z = torch.zeros(h, D, dtype=torch.float64, device=q.device)
        return z, torch.full((h,), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0]
    s = scale * (q @ k.T)
    ds = (2.0 ** -19 * abs(scale) * (q.abs() @ k.abs().T) + 2.0 ** -22 * s.abs()).amax(1)
    top = s.amax(1, keepdim=True)
    w = torch.exp(s - top)
    total = w.sum(1, keepdim=True)
    o, mag = (w @ v) / total, (w @ v.abs()) / total
    lse = (top + total.log())[:, 0]
    sums = (n / 128 + 64) * 2.0 ** -22
    return o, lse, (2 * ds[:, None] + 2.0 ** -21 + sums) * mag, ds + sums + 2.0 ** -22 * lse.abs()


def check(got, ref, tol, what):
    got = got.double()
    assert torch.isfinite(got).all() or not torch.isfinite(ref).all(), f"{what}: not finite"
    bad = ~((got - ref).abs() <= tol) & (got != ref)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, the worst by "
                           f"{float(((got - ref).abs() / tol)[bad].max()):.3g} tolerances")


def check_rows(out, lse, q, k, v, scale, what):
    """One row's outputs [h, D] and lse [h] against the reference."""
    o, l, to, tl = attend_ref(q, k, v, scale)
    check(out, o, to + (2.0 ** -8 * o.abs() if out.dtype == torch.bfloat16 else 0), what)
    check(lse, l, tl, what + " lse")


def status_ok():
    torch.cuda.synchronize()
    assert hhr.hhr_read_device_status() == (hhr.HHR_OK, 0)
