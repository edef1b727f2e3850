"""Latent attention where the range of the numbers decides: FP8 pages whose rows differ much in
scale or weight, bounds of FP8 decode from its own arithmetic, large softcaps, tiny rows."""
import math

import pytest
import torch

from latent_harness import (BF16, F64, H_BF16, H_E4M3, NOPE, PAGE, R, THETA, EPS, V, LatentLayer, Pages, attend, check,
                            check_attention, cu, gen, i32, no_error, randn)
from paged_sliding_window_gb300 import binding
from test_gpu_latent import P_ERR, P_ERR_PREFILL, S_ERR, _decode_call, _decode_inputs, _decode_ref

pytestmark = pytest.mark.gpu

# FP8 pages. P times the row's scale is taken in three E4M3 parts, each 16 times finer than the one
# before: off by 2^-12 of itself, or where the last part is subnormal by 2^-10 / 256 of the unit in
# use, in which the largest of a tile's 64 rows is 2^-4 or more: 64 * 2^-18 / 2^-4 of their sum;
# or less, where all that it loses is 2^-9 of the probability at most
P_ERR8 = 2.0 ** -12 + 2.0 ** -8


def fp8_scores(layer, q, rows, mag):
    """mag, raised by what the query's two E4M3 parts leave: the codes of q 2^k with the largest of
    a head in [128, 256) are exact but where the second part is subnormal: 2^-10 / 16 there, 2^-21
    of the largest; a score is off by that times sum |k_d|."""
    amax = q.to(F64).abs().amax(-1)
    return mag + (layer.scale * amax * 2.0 ** -21 * rows.abs().sum(1).amax() / S_ERR)[:, None]


def check_decode(layer, pg, q, lens, out, lse, what, p_err=None):
    for b, n in enumerate(lens):
        o, l, a, m = _decode_ref(layer, pg, q, b, n)
        p = P_ERR
        if pg.fp8:
            m, p = fp8_scores(layer, q[b], pg.rows(b, 0, n), m), p_err or P_ERR8
        check_attention(out[b][:, None], lse[b][:, None], (o, l, a, m), p, S_ERR, f"{what}, sequence {b} of {n}")


def run_decode(layer, pg, q, lens, what, p_err=None):
    n, H, L = len(lens), layer.n_heads, layer.latent_dim
    out, lse = torch.full((n, H, L), float("nan"), dtype=BF16, device="cuda"), torch.full((n, H), float("nan"), device="cuda")
    _decode_call(layer, pg, q, i32(lens), out, lse, binding.alloc_latent_workspace(layer, n))
    no_error()
    check_decode(layer, pg, q, lens, out, lse, what, p_err)
    return out, lse


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("L,H,lens,grow,scale", [(256, 4, [1500, 300], 2.0, 1.0), (512, 16, [3000, 129], 0.0, 1.0),
                                                 (512, 16, [3000, 129], 0.0, 1e-4), (512, 24, [700, 65], 0.3, 0.3)])
def test_decode_bounds(L, H, lens, grow, scale, fp8):
    """Growing, peaked and flat scores within bounds that are as tight on FP8 pages as on bf16
    pages but for P's parts."""
    layer = LatentLayer(H, L, scale=scale)
    pg, q = _decode_inputs(layer, lens, fp8, 5, grow=grow)
    run_decode(layer, pg, q, lens, "bounds")


def sink_inputs(layer, lens, bits, ratio, seed, at=0):
    """Rows of equal scores behind one (row `at`) whose score is `bits` powers of two above theirs and
    whose row scale is `ratio` times theirs; its latent is small, as that of such a row mostly is."""
    g, L, H = gen(seed), layer.latent_dim, layer.n_heads
    pg = Pages(lens, L, True, seed)
    q = torch.zeros(len(lens), H, L + R, device="cuda")
    q[..., L] = 512.0  # (its codes are exact, and the outlier's score needs no large value)
    for b, n in enumerate(lens):
        rows = 1 + 0.25 * randn(g, n, L + R)
        rows[:, L] = 0.0
        rows[at] *= 0.125
        rows[at, L] = bits * math.log(2.0) / (512.0 * layer.scale)
        rows[at, L + 1] = 3.5 * ratio
        pg.put(b, rows)
    return pg, q.to(BF16)


@pytest.mark.parametrize("L,H,lens", [(512, 16, [4000] * 160), (512, 24, [4000, 130]), (256, 32, [3001] * 160), (256, 3, [64, 65, 1000])])
@pytest.mark.parametrize("bits,ratio,at", [(14, 256.0, 0), (10, 4096.0, 0), (17, 1.0, 0), (14, 256.0, 40), (12, 64.0, 63)])
def test_decode_fp8_rows_behind_an_outlier(L, H, lens, bits, ratio, at):
    """What follows a row of large score and large scale weighs as much as it should, although each
    of its weights times its scale is 2^-17 to 2^-23 of the outlier's. (The unit moves to the tiles
    behind the outlier's, whose largest weight is then 4 units or more; all that the other rows of
    its own tile weigh may be lost.)"""
    layer = LatentLayer(H, L, scale=0.01)
    pg, q = sink_inputs(layer, lens, bits, ratio, 31, at)
    out, lse = torch.empty(len(lens), H, L, dtype=BF16, device="cuda"), torch.empty(len(lens), H, device="cuda")
    _decode_call(layer, pg, q, i32(lens), out, lse, binding.alloc_latent_workspace(layer, len(lens)))
    no_error()
    for b, n in list(enumerate(lens))[::80] + [(len(lens) - 1, lens[-1])]:
        o, l, a, m = _decode_ref(layer, pg, q, b, n)
        # the outlier's tile: at most 63 rows, all of whose weight may be lost
        own = min(63, n - 1) / (2.0 ** bits + n - 1)
        rows = pg.rows(b, 0, n)
        lost = own * rows[:64, :L].abs().amax(0)
        e = m * S_ERR
        check(out[b][:, None], o, H_BF16 * o.abs() * 1.01 + a * (2.0 ** -11 + 3 * e + 2.0 ** -18)[..., None] + 1.01 * lost + 1e-30,
              f"out, sequence {b} of {n}")
        check(lse[b][:, None], l, 1.2 * e + 2.0 ** -20 * (l.abs() + 4), f"lse, sequence {b} of {n}")


@pytest.mark.parametrize("H,L,cap", [(16, 512, 0.0), (32, 512, 0.0), (9, 256, 60.0)])
def test_decode_fp8_levels(H, L, cap):
    """Tiles whose scores and row scales go up and down by many powers of two, zero rows and a zero
    first tile among them."""
    layer = LatentLayer(H, L, scale=0.02, softcap=cap)
    lens = [3000, 64, 777, 1]
    g, pg = gen(17), Pages(lens, L, True, 17)
    q = (0.2 * randn(g, len(lens), H, L + R)).to(BF16)
    q[..., L] = 16.0
    for b, n in enumerate(lens):
        rows = randn(g, n, L + R)
        tiles = -(-n // 64)
        level = (torch.rand(tiles, generator=g, device="cuda") * 40 - 30).repeat_interleave(64)[:n]
        size = torch.exp2(torch.rand(tiles, generator=g, device="cuda") * 24 - 18).repeat_interleave(64)[:n]
        rows *= size[:, None]
        rows[:, L] = level / (16.0 * layer.scale)
        if b % 2 == 0:
            rows[:64] = 0
        rows[::5] = 0
        pg.put(b, rows)
    run_decode(layer, pg, q, lens, "levels")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("cap", [1e3, 1e6, 1e30])
def test_decode_large_softcap(cap, fp8):
    """A cap far above the scores leaves them as they are."""
    layer, lens = LatentLayer(16, 512, scale=0.07, softcap=cap), [700, 65]
    pg, q = _decode_inputs(layer, lens, fp8, 5)
    run_decode(layer, pg, q, lens, f"softcap {cap}")


@pytest.mark.parametrize("cap", [1e3, 1e6, 1e30])
@pytest.mark.parametrize("H,new,past", [(2, [200, 64], [300, 0]), (2, [520], [100]), (90, [150, 30], [100, 0])], ids=["split", "pair", "single"])
def test_prefill_large_softcap(H, new, past, cap):
    layer, g = LatentLayer(H, scale=0.07, softcap=cap), gen(3)
    keys, T = [n + p for n, p in zip(new, past)], sum(new)
    q = randn(g, T, H, NOPE + R).to(BF16)
    kv, rope = randn(g, sum(keys), H, NOPE + V).to(BF16), randn(g, sum(keys), R).to(BF16)
    out, lse = torch.empty(T, H, V, dtype=BF16, device="cuda"), torch.empty(T, H, device="cuda")
    binding.attn_prefill_latent(layer, q, cu(new), i32(past), max(new), kv, rope, cu(keys), out, lse)
    no_error()
    q0 = k0 = 0
    for n, p, t in zip(new, past, keys):
        k = torch.cat([kv[k0:k0 + t, :, :NOPE], rope[k0:k0 + t, None].expand(-1, H, -1)], -1)
        ref = attend(q[q0:q0 + n].to(F64).transpose(0, 1), k.to(F64).transpose(0, 1), kv[k0:k0 + t, :, NOPE:].to(F64).transpose(0, 1),
                     p + torch.arange(n, device="cuda"), torch.arange(t, device="cuda"), layer)
        check_attention(out[q0:q0 + n].transpose(0, 1), lse[q0:q0 + n].transpose(0, 1), ref, P_ERR_PREFILL, S_ERR, f"softcap {cap}")
        q0, k0 = q0 + n, k0 + t


def test_write_fp8_tiny_rows():
    """Rows so small that 448 / amax has no fp32 value are zero rows; somewhat larger ones are
    rows like any other. None becomes NaN."""
    L, n = 256, 40
    layer, g, pg = LatentLayer(1, L), gen(2), Pages([n, n, n], L, True, 2)
    ckv = randn(g, n, L + R).to(BF16)
    ckv[:, L:] = 0
    ckv[:, :8] = 0
    want0 = ckv[:, :L].to(F64)
    want0 = want0 / (want0.square().mean(1, keepdim=True) + EPS).sqrt()
    for b, size in enumerate((2.0 ** -100, 2.0 ** -115, 2.0 ** -122)):
        w = torch.full((L,), size, device="cuda")
        table = pg.table[b:b + 1].contiguous()
        binding.latent_norm_rope_cache_write_fp8(layer, binding.make_latent_norm(THETA, EPS, w), ckv, None, cu([n]), i32([0]),
                                                 binding.make_pages(table, pg.blocks), None, pg.pool, pg.scale)
        no_error()
        got, sc = pg.rows(b, 0, n), pg.scale.view(-1)[pg.slots(b, 0, n)].to(F64)[:, None]
        want = torch.cat([want0 * size, torch.zeros(n, R, dtype=F64, device="cuda")], 1)
        if size < 2.0 ** -121:
            assert bool((got == 0).all()) and bool((sc == 0).all())
        else:
            check(got, want, (H_E4M3 + 2.0 ** -17) * want.abs() + 2.0 ** -10 * sc, f"rows of {size}")
