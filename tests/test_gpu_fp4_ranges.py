"""The 4-bit operators where their arithmetic is at its edges: queries of very different size in one group,
tensor scales that are no power of two, quotients on and beside the borders between codes."""
import functools

import numpy as np
import pytest
import torch

from fp4_harness import BF16, GRID, Cache, Layer, cu, gen, i32, no_error, normed, quantised, randn
from paged_sliding_window_gb300 import binding
from test_gpu_fp4 import compare, decode

pytestmark = pytest.mark.gpu

# Powers of two of the heads of a group, no two alike: scores from far apart to all the same, the
# last but two with every value below 2^-112, where the queries' own scaling has its end.
SIZES = (0, -3, 2, -5, -118, 1, -60, -1)


@pytest.mark.parametrize("layer", [Layer(16, 2, 256, scale=0.25), Layer(5, 1, 256, scale=0.25, softcap=20.0), Layer(22, 2, 256, scale=0.25, k_eq_v=True),
                                   Layer(8, 1, 512, scale=0.25), Layer(16, 2, 512, scale=0.25, k_eq_v=True)],
                         ids=["256", "256-g5-softcap", "256-g11-keqv", "512", "512-keqv"])
def test_heads_of_different_size(layer):
    """Every head has a query of its own and a size of its own, and so weights of its own: from one key
    that takes nearly all of them to equal ones."""
    lens, g = [700, 33, 1], gen(60)
    cache, n = Cache(layer, lens, 60), sum(lens)
    k = normed(g, n, layer.n_kv_heads, layer.head_dim)
    v = None if layer.k_eq_v else randn(g, *k.shape).to(BF16)
    cache.write(k, v, lens, [0] * len(lens))
    size = torch.tensor([2.0 ** SIZES[h % len(SIZES)] for h in range(layer.n_q_heads)], dtype=torch.float64, device="cuda")
    q = (randn(g, len(lens), layer.n_q_heads, layer.head_dim).to(torch.float64) * size[:, None]).to(BF16)
    got = decode(layer, cache, q, lens)
    no_error()
    compare(layer, cache, q, lens, got)


def test_heads_of_different_size_can_be_told_apart():
    """Had two heads each other's factor, their results would differ by far more than the bounds."""
    layer, lens, g = Layer(8, 1, 256, scale=0.25), [400], gen(61)
    cache = Cache(layer, lens, 61)
    k = normed(g, 400, 1, 256)
    cache.write(k, k, lens, [0])
    q = randn(g, 1, 1, 256).expand(-1, 8, -1) * torch.tensor([2.0 ** e for e in SIZES], device="cuda")[:, None]
    got = decode(layer, cache, q.to(BF16).contiguous(), lens)
    no_error()
    compare(layer, cache, q.to(BF16), lens, got)
    order = sorted((e, h) for h, e in enumerate(SIZES) if e >= -5)
    lse = got[1][0]
    assert all(float(lse[b] - lse[a]) > 0.01 for (_, a), (_, b) in zip(order, order[1:]))


@pytest.mark.parametrize("layer", [Layer(2, 2, 256), Layer(1, 1, 512)], ids=["256", "512"])
def test_write_tensor_scales_of_all_kinds(layer):
    """Every value is the one of the format's definition, whatever the tensor scale: y has then all of
    its 24 bits."""
    g, n = gen(62), 64
    rng = np.random.RandomState(62)
    scales = [0.37, 2.5, 1 / 3, 0.1, 1.0000001, 1.9999999, 2.0 ** -60, 2.0 ** 60, *(2.0 ** rng.uniform(-6, 6, 40)), *(2.0 ** rng.uniform(-59, 59, 12))]
    for gs, other in zip(scales, scales[::-1]):
        cache = Cache(layer, [n], 63, spare=0)
        x = [(normed(g, n, layer.n_kv_heads, layer.head_dim).float() * s * 2.0 ** torch.randint(-8, 9, (n, 1, 1), device="cuda", generator=g)).to(BF16)
             for s in (gs, other)]
        cache.write(*x, [n], [0], (gs, other))
        for rows, pool, s in zip(x, (cache.k, cache.v), (gs, other)):
            assert torch.equal(cache.rows(pool, 0, 0, n, s), quantised(rows, s)), s
    no_error()


# ---------------------------------------------------------------- quotients at the codes' borders

MIDDLES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


@functools.lru_cache(maxsize=1)
def border_cases():
    """(significand m of a block's scale, border, steps from it, x, gs): x bf16 and a tensor scale whose
    reciprocal times x is, in fp32, `steps` steps of fp32 from border * m. Found by trying every
    significand of bf16 with the reciprocals next to the wanted one."""
    one = np.float32(1)
    sig = (np.arange(128, 256) / 128).astype(np.float32)  # of bf16
    cases = []
    for m in range(8, 16):
        for border in MIDDLES:
            for steps in (-1, 0, 1):
                y = np.float32(border * m / 8)
                y = np.nextafter(y, np.float32(100 * steps), dtype=np.float32) if steps else y
                hits = []
                for x in sig:
                    want = np.float32(y / x)
                    for inv in (np.nextafter(want, np.float32(0)), want, np.nextafter(want, np.float32(100))):
                        if np.float32(x * inv) != y:
                            continue
                        near = np.float32(one / inv)
                        for gs in (np.nextafter(near, np.float32(0)), near, np.nextafter(near, np.float32(100))):
                            if np.float32(one / gs) == inv:
                                hits.append((float(x), float(gs)))
                                break
                assert hits, (m, border, steps)
                pick = np.random.RandomState(len(cases)).permutation(len(hits))[:3]
                cases += [(m, border, steps, *hits[i]) for i in pick]
    return cases


def border_rows(case, hd):
    """One row of hd values: in its blocks of 16, one for every exponent at which the scale m 2^j is an
    E4M3 number, the value that sets the scale, then x and -x. And the scales ([hd / 16], 0: none)."""
    m, border, steps, x, gs = case
    inv = np.float32(1) / np.float32(gs)
    rows, scales = np.zeros((hd // 16, 16)), np.zeros(hd // 16)
    at = [j for j in range(-9, 9) if (m / 8 * 2.0 ** j * 512) % 1 == 0 and m / 8 * 2.0 ** j <= 448]
    for i, j in enumerate(at[:hd // 16]):
        rows[i, :3] = 6 * m / 8 / float(inv) * 2.0 ** j, x * 2.0 ** j, -x * 2.0 ** j
        scales[i] = m / 8 * 2.0 ** j
    return rows.reshape(hd), scales


@pytest.mark.parametrize("hd", [256, 512])
def test_write_on_and_beside_the_borders_between_codes(hd):
    """y / s on a border and one step of fp32 to either side of it, at every scale that E4M3 has: the code
    is the one that the quotient in 64 bits gives, and the one of an ordinary division in fp32."""
    layer, cases = Layer(1, 1, hd), border_cases()
    grid, mid = torch.tensor(GRID, device="cuda"), torch.tensor(MIDDLES, device="cuda")
    seen, room = set(), hd // 16
    for a, b in zip(cases[::2], cases[1::2]):
        cache = Cache(layer, [1], 64, spare=0)
        both = [border_rows(c, hd) for c in (a, b)]
        x = [torch.tensor(r, device="cuda").to(BF16).view(1, 1, hd) for r, _ in both]
        binding.kv_cache_write_fp4(layer, *x, cu([1]), i32([0]), cache.pages, cache.k, cache.v, k_scale=a[4], v_scale=b[4])
        for case, row, pool, (_, scales) in zip((a, b), x, (cache.k, cache.v), both):
            m, border, steps, _, gs = case
            got = cache.rows(pool, 0, 0, 1, gs)
            assert torch.equal(got, quantised(row, gs)), case
            s = torch.tensor(scales, dtype=torch.float32, device="cuda")
            have = s > 0
            inv = torch.tensor(1.0, device="cuda") / torch.tensor(gs, dtype=torch.float32, device="cuda")
            y = (row.float() * inv).view(-1, 16)[have, 1:3]
            wanted = np.float32(border * m / 8)
            wanted = np.nextafter(wanted, np.float32(100 * steps), dtype=np.float32) if steps else wanted
            power = s[have] / (m / 8)  # (of two)
            assert bool((y[:, 0] / power == float(wanted)).all()) and torch.equal(y[:, 1], -y[:, 0]), case
            quot = y.abs() / s[have, None]
            code = torch.searchsorted(mid, quot.contiguous())
            code = torch.where(code % 2 == 1, torch.searchsorted(mid, quot.contiguous(), right=True), code)
            want = torch.copysign(grid[code], y).double() * s[have, None].double() * float(np.float32(gs))
            assert torch.equal(got.view(-1, 16)[have, 1:3], want), case
            seen |= set(s.tolist()) - {0.0}
    no_error()
    # all positive scales that E4M3 has, 126, but for those that a row has no block for
    every = [sum((m / 8 * 2.0 ** j * 512) % 1 == 0 and m / 8 * 2.0 ** j <= 448 for j in range(-9, 9)) for m in range(8, 16)]
    assert sum(every) == 126 and len(seen) == sum(min(room, n) for n in every)
