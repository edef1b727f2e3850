"""Plain 64-bit implementations of the latent-attention operators, and inputs
for them, for the parity tests. Every pool starts as NaN (bf16) or NaN codes
and NaN scales (FP8), so any slot that a kernel should not read shows."""
import math

import numpy as np
import torch

from paged_sliding_window_gb300 import binding
from paged_sliding_window_gb300.workloads import LatentLayer  # noqa: F401

R, NOPE, V, PAGE = 64, 128, 128, 16
F64, BF16 = torch.float64, torch.bfloat16
THETA, EPS = 10000.0, 1e-6
# half a rounding step relative to the value
H_BF16, H_E4M3 = 2.0 ** -8, 2.0 ** -4


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def cu(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]))


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


class Pages:
    """A pool whose pages go to sequences of the given lengths in random order."""

    def __init__(self, lens, L, fp8, seed, spare=3):
        g = gen(seed)
        n = [-(-int(x) // PAGE) for x in lens]
        self.blocks, self.L, self.fp8 = sum(n) + spare, L, fp8
        perm = torch.randperm(self.blocks, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((max(1, len(n)), max([1] + n)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, k in enumerate(n):
            self.table[b, :k] = perm[at:at + k]
            at += k
        shape = (self.blocks, PAGE, L + R)
        if fp8:
            self.pool = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
            self.scale = torch.full(shape[:2], float("nan"), device="cuda")
        else:
            self.pool = torch.full(shape, float("nan"), dtype=BF16, device="cuda")
            self.scale = None
        self.pages = binding.make_pages(self.table, self.blocks)

    def slots(self, b, lo, hi):
        pos = torch.arange(lo, hi, device="cuda")
        return self.table[b].long()[pos // PAGE] * PAGE + pos % PAGE

    def put(self, b, rows):
        """Rows (float) of sequence b from position 0 on, stored as the pool's type."""
        at = self.slots(b, 0, rows.shape[0])
        if self.fp8:
            amax = rows.float().abs().amax(1, keepdim=True)
            k = torch.where(amax > 0, 448.0 / amax, torch.zeros_like(amax))
            self.pool.view(-1, self.L + R)[at] = (rows.float() * k).to(torch.float8_e4m3fn).view(torch.uint8)
            self.scale.view(-1)[at] = amax[:, 0] / 448.0
        else:
            self.pool.view(-1, self.L + R)[at] = rows.to(BF16)

    def rows(self, b, lo, hi):
        """What the slots stand for, in 64 bits."""
        at = self.slots(b, lo, hi)
        x = self.pool.view(-1, self.L + R)[at]
        if self.fp8:
            return x.view(torch.float8_e4m3fn).to(F64) * self.scale.view(-1, 1)[at].to(F64)
        return x.to(F64)


def attend(q, k, v, p, pos, layer):
    """q [h, n, d] at positions p [n] over k, v [h or 1, t, .] at positions pos [t]: out, lse,
    the weighted mean of |v| and the largest sum of |scale q_d k_d| of each row (for tolerances)."""
    h = q.shape[0]
    k, v = k.expand(h, -1, -1), v.expand(h, -1, -1)
    x = layer.scale * torch.matmul(q, k.transpose(1, 2))
    mag = layer.scale * torch.matmul(q.abs(), k.abs().transpose(1, 2))
    if layer.softcap:
        x = layer.softcap * torch.tanh(x / layer.softcap)
    seen = pos[None, :] <= p[:, None]
    if layer.window:
        seen &= p[:, None] - pos[None, :] < layer.window
    if k.shape[1] == 0:
        z = q.new_zeros(h, q.shape[1], v.shape[2])
        return z, torch.full(z.shape[:2], -math.inf, dtype=F64, device=q.device), z, z[..., 0]
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = (x - m).exp()
    l = e.sum(-1, keepdim=True)
    w = e / torch.where(l == 0, torch.ones_like(l), l)
    return (torch.matmul(w, v), (l.log() + m)[..., 0], torch.matmul(w, v.abs()),
            mag.masked_fill(~seen, 0.0).amax(-1))


def check(got, ref, bound, what):
    got, ref = got.to(F64), ref.to(F64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    off = torch.where(inf, torch.zeros_like(ref), (got - ref).abs())
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float(torch.nan_to_num(off / bound, nan=1e9).max()):.3g} of it, first at "
                           f"{bad.nonzero()[0].tolist()}: got {got[tuple(bad.nonzero()[0])]:.8g}, "
                           f"want {ref[tuple(bad.nonzero()[0])]:.8g}")


def check_attention(out, lse, ref, p_err, s_err, what):
    """Bounds of an attention result. The kernel's weights are off by at most p_err (relative:
    the rounding of P) and by the scores' errors, s_err * (sum of |scale q_d k_d|), once in the
    numerator and once in the sum; exp, the sums and the division add a few fp32 steps (2^-18
    covers 64). The result is rounded once, to bf16."""
    o, l, absv, mag = ref
    e = (mag * s_err).clamp(max=0.25)
    check(out, o, H_BF16 * o.abs() * 1.01 + absv * (p_err + 3 * e + 2.0 ** -18)[..., None] + 1e-30, what + " out")
    if lse is not None:
        finite = torch.where(torch.isinf(l), torch.zeros_like(l), l)
        check(lse, l, 1.2 * e + 2.0 ** -20 * (finite.abs() + 4), what + " lse")


def rotated(x, pos):
    """Rotate-half of [n, ..., 64] at positions pos [n] in 64 bits."""
    i = torch.arange(R // 2, device="cuda", dtype=F64)
    a = pos.to(F64)[:, None] * THETA ** (-2 * i / R)
    a = a.view(a.shape[0], *[1] * (x.dim() - 2), R // 2)
    lo, hi = x[..., :R // 2].to(F64), x[..., R // 2:].to(F64)
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)


def row_of(ckv, pos, L, weight):
    c = ckv[:, :L].to(F64)
    c = c / (c.square().mean(1, keepdim=True) + EPS).sqrt()
    if weight is not None:
        c = c * weight.to(F64)
    return torch.cat([c, rotated(ckv[:, L:], pos)], 1)


def rot_mag(x):
    """|x_i| + |x_partner|: what a rotation's fp32 errors are relative to."""
    a = x.to(F64).abs()
    return torch.cat([a[..., :R // 2] + a[..., R // 2:]] * 2, -1)


def no_error():
    torch.cuda.synchronize()
    got = binding.get_error()
    assert got == 0, f"error word {got}"


def takes_error(bits):
    torch.cuda.synchronize()
    got = binding.get_error()
    assert got == bits, f"error word {got}, want {bits}"
