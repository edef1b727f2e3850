"""Plain 64-bit implementations of the 4-bit pages' format and operators, for
the parity tests. Every pool starts with codes of 0xFF and scales that are NaN,
so any slot that a kernel should not use shows."""
import numpy as np
import torch

from latent_harness import BF16, F64, attend, check, cu, gen, i32, no_error, randn, takes_error  # noqa: F401
from paged_sliding_window_gb300 import binding
from paged_sliding_window_gb300.workloads import Layer  # noqa: F401

PAGE = 16
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# What a decode's weights and scores may be off by. P = 2^(z - m) is rounded once, to fp16: by half a
# step, 2^-11 of it, or by 2^-25 where it is below 2^-14. As m is at least 6 below the largest z, the sum
# of P is at least 2^6, so the second adds at most 2^-25 / 2^6 |v_j| for every key j to a result:
# P_ABS * sum |v_j|. A score: q in fp16 is exact but for 2^-39 of the head's largest, K's codes times
# scales are exact in fp16; 32 products of 16 terms are summed in fp32, each step off by at most 17
# units of 2^-24 of what is summed so far (32 * 17 * 2^-24 < 2^-14).
P_ERR = 2.0 ** -11 + 2.0 ** -15
P_ABS = 2.0 ** -31
S_ERR = 2.0 ** -14
H_BF16 = 2.0 ** -8  # half a step of the result


def places(hd, device="cuda"):
    """[16, hd] byte and half (0 low, 1 high) of every code of a page, [16, hd / 16] byte of every scale."""
    code, half, scale = np.zeros((PAGE, hd), np.int64), np.zeros((PAGE, hd), np.int64), np.zeros((PAGE, hd // 16), np.int64)
    for r in range(PAGE):
        for d in range(hd):
            unit = d % 256 // 32
            code[r, d] = d // 256 * 2048 + r * 128 + (unit ^ (r & 7)) * 16 + d % 32 // 2
            half[r, d] = d & 1
        for k in range(hd // 16):
            c, t, e = k // 8, k // 2 % 4, k % 2
            if hd == 512:
                c = 2 * (c % 2) + c // 2
            scale[r, k] = 8 * hd + r * (hd // 16) + t * (hd // 64) + 2 * c + e
    t = lambda a: torch.tensor(a, device=device)  # noqa: E731
    return t(code), t(half), t(scale)


def quantised(x, gs):
    """The values [..., hd] that rows x stand for, in 64 bits, from the format's definition (its steps up
    to y / s are fp32; the nearest code is found by comparing with the middles, which are exact)."""
    inv = torch.tensor(1.0, device=x.device) / torch.tensor(gs, dtype=torch.float32, device=x.device)
    y = torch.nan_to_num(x.float() * inv, nan=4096.0).clamp(-4096, 4096).unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1, keepdim=True) * torch.tensor(1 / 6, dtype=torch.float32)).clamp(max=448).to(torch.float8_e4m3fn).to(F64)
    a = y.to(F64).abs() / torch.where(s == 0, torch.ones_like(s), s)
    grid = torch.tensor(GRID, dtype=F64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    code = torch.searchsorted(mid, a.contiguous())            # ties go down ...
    up = torch.searchsorted(mid, a.contiguous(), right=True)  # ... or up: to the even code
    code = torch.where(code % 2 == 1, up, code)
    return (torch.copysign(grid[code], y.to(F64)) * s * float(np.float32(gs))).flatten(-2)


def unpack(pool, hd, gs):
    """[blocks, heads, 9 hd] -> [blocks, heads, 16, hd] in 64 bits."""
    code, half, scale = places(hd, pool.device)
    c = pool[..., code].int() >> (4 * half) & 15
    grid = torch.tensor(GRID, dtype=F64, device=pool.device)
    s = pool[..., scale].view(torch.float8_e4m3fn).to(F64)
    v = torch.where(c >= 8, -grid[c & 7], grid[c & 7])
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2) * float(np.float32(gs))


def empty_pool(layer, blocks):
    pool = binding.alloc_fp4_pool(layer, blocks)
    pool.fill_(0xFF)
    pool[..., 8 * layer.head_dim:] = 0x7F
    return pool


class Cache:
    """4-bit pools whose pages go to sequences of the given lengths in random order."""

    def __init__(self, layer, lens, seed, spare=3, width=None):
        g = gen(seed)
        self.layer, n = layer, [-(-int(x) // PAGE) for x in lens]
        self.blocks = sum(n) + spare
        perm = torch.randperm(self.blocks, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((max(1, len(n)), width or max([1] + n)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, k in enumerate(n):
            self.table[b, :k] = perm[at:at + k]
            at += k
        self.pages = binding.make_pages(self.table, self.blocks)
        self.k = empty_pool(layer, self.blocks)
        self.v = None if layer.k_eq_v else empty_pool(layer, self.blocks)

    def write(self, k, v, new, past, gs=(1.0, 1.0), stream=None):
        binding.kv_cache_write_fp4(self.layer, k, v, cu(new), i32(past), self.pages, self.k, self.v,
                                   k_scale=gs[0], v_scale=gs[1], stream=stream)

    def rows(self, pool, b, lo, hi, gs):
        """Positions [lo, hi) of sequence b, [hi - lo, n_kv, hd] in 64 bits."""
        pos = torch.arange(lo, hi, device="cuda")
        page = self.table[b].long()[pos // PAGE]
        used, at = torch.unique(page, return_inverse=True)
        return unpack(pool[used], self.layer.head_dim, gs)[at, :, pos % PAGE]


def check_decode(out, lse, ref, what):
    """Bounds of a decode [heads, hd]: the weights' and the scores' errors (once in the numerator, once in
    the sum; 2^-18 covers the exponential, the sums and the division), one rounding to bf16."""
    o, l, absv, mag, all_v = ref
    e = (mag * S_ERR).clamp(max=0.25)
    check(out, o, H_BF16 * o.abs() * 1.01 + absv * (P_ERR + 3 * e + 2.0 ** -18)[:, None] + 1.01 * P_ABS * all_v, what + " out")
    if lse is not None:
        check(lse, l, 1.2 * e + 2.0 ** -20 * (l.abs() + 4), what + " lse")


def decode_ref(layer, cache, q, b, n, gs=(1.0, 1.0), zero=()):
    """Attention of sequence b of n keys: per query head, (out, lse, weighted |v|, magnitude of a score,
    sum of |v|). zero: positions whose rows are zeros."""
    lo = max(0, n - layer.window) if layer.window else 0
    k = cache.rows(cache.k, b, lo, n, gs[0])
    v = k if layer.k_eq_v else cache.rows(cache.v, b, lo, n, gs[1])
    if len(zero):
        k, v = k.clone(), v.clone()
        for p in zero:
            k[p - lo], v[p - lo] = 0, 0
    G = layer.n_q_heads // layer.n_kv_heads
    k, v = (x.transpose(0, 1).repeat_interleave(G, 0) for x in (k, v))
    ref = attend(q[b].to(F64)[:, None], k, v, torch.tensor([n - 1], device="cuda"), torch.arange(lo, n, device="cuda"), layer)
    return (*(x[:, 0] for x in ref), v.abs().sum(1))


def normed(g, *shape):
    x = randn(g, *shape)
    return (x / x.square().mean(-1, keepdim=True).sqrt()).to(BF16)
