"""The 4-bit pages' operators against plain implementations in 64 bits."""
import math

import pytest
import torch

from fp4_harness import (BF16, F64, PAGE, Cache, Layer, check, check_decode, cu, decode_ref,
                         empty_pool, gen, i32, no_error, normed, quantised, randn, takes_error, unpack)
from paged_sliding_window_gb300 import binding

pytestmark = pytest.mark.gpu

L256, L512 = Layer(4, 2, 256), Layer(8, 2, 512, scale=0.05)
KEQV = Layer(6, 3, 512, k_eq_v=True, scale=0.1)


def rows_of(kind, g, n, layer):
    shape = (n, layer.n_kv_heads, layer.head_dim)
    if kind == "normed":
        return normed(g, *shape)
    if kind == "wide":  # magnitudes over the whole range and beyond both ends
        return (randn(g, *shape) * 2.0 ** torch.randint(-14, 15, (*shape[:2], shape[2] // 16, 1), device="cuda", generator=g).float()
                .expand(-1, -1, -1, 16).flatten(-2)).to(BF16)
    # ties: multiples of the middles of the grid times scales with few bits
    grid = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0], device="cuda")
    x = grid[torch.randint(0, 15, shape, device="cuda", generator=g)] * torch.where(torch.rand(shape, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    x[..., ::16] = 6.0  # the block's scale is then the factor
    f = torch.tensor([1.0, 1.125, 1.25, 1.375, 1.5, 1.625, 1.75, 1.875], device="cuda")[torch.randint(0, 8, (*shape[:2], shape[2] // 16, 1), device="cuda", generator=g)]
    return (x.unflatten(-1, (-1, 16)) * f).flatten(-2).to(BF16)


# ---------------------------------------------------------------- write and read-back

@pytest.mark.parametrize("kind", ["normed", "wide", "ties"])
@pytest.mark.parametrize("layer,new,past,gs", [
    pytest.param(L256, [1], [0], (1.0, 1.0), id="one-token"),
    pytest.param(L256, [3, 0, 17, 1, 40], [15, 4, 0, 16, 31], (1.0, 1.0), id="ragged"),
    pytest.param(Layer(1, 1, 256), [33, 2], [5, 100], (0.25, 4.0), id="one-head"),
    pytest.param(Layer(5, 5, 512), [20, 1], [3, 15], (2.0, 0.5), id="five-heads-512"),
    pytest.param(KEQV, [50, 0, 7], [2, 9, 64], (1.0, 1.0), id="keqv"),
    pytest.param(L512, [1] * 300, list(range(300)), (1.0, 1.0), id="300-sequences"),
])
def test_write(layer, new, past, gs, kind):
    """Every written value is the nearest the format has (powers of two as tensor scales: then the steps
    in front of the division are exact), every other byte of the pools stays."""
    g, n = gen(1), sum(new)
    cache = Cache(layer, [a + b for a, b in zip(new, past)], 2)
    k = rows_of(kind, g, n, layer)
    v = None if layer.k_eq_v else rows_of(kind, g, n, layer)
    cache.write(k, v, new, past, gs)
    no_error()
    written = torch.zeros(cache.blocks, PAGE, dtype=torch.bool, device="cuda")
    t = 0
    for b, (m, p) in enumerate(zip(new, past)):
        pos = torch.arange(p, p + m, device="cuda")
        blk = cache.table[b].long()[pos // PAGE]
        written[blk, pos % PAGE] = True
        for x, pool, s in ((k, cache.k, gs[0]), (v, cache.v, gs[1])):
            if x is not None and m:
                assert torch.equal(cache.rows(pool, b, p, p + m, s), quantised(x[t:t + m], s)), (b, s)
        t += m
    for pool in (cache.k, cache.v):
        if pool is not None:  # untouched rows: the scales are still NaN, the codes -6
            rest = unpack(pool, layer.head_dim, 1.0).transpose(1, 2)[~written]
            assert bool(rest.isnan().all())
            fresh = empty_pool(layer, 1)
            codes = pool[..., :8 * layer.head_dim].view(-1, layer.n_kv_heads, layer.head_dim // 256, PAGE, 128)
            assert bool((codes.permute(0, 3, 1, 2, 4)[~written] == fresh[0, 0, 0]).all())


def test_write_any_tensor_scale():
    """A tensor scale that is no power of two: at most one step of the grid from the nearest value in 64
    bits, and that only where y / s lies within 2^-22 of a middle."""
    g, layer, gs = gen(3), L256, 0.37
    cache = Cache(layer, [200], 4)
    k = normed(g, 200, 2, 256)
    cache.write(k, k, [200], [0], (gs, gs))
    no_error()
    got, want = cache.rows(cache.k, 0, 0, 200, gs), quantised(k, gs)
    assert torch.equal(cache.k, cache.v)
    assert float((got != want).float().mean()) < 1e-5


def test_write_no_finite_value():
    """Infinities and NaN become the ends of the range; zero rows and rows too small are zeros."""
    layer, cache = L256, Cache(L256, [16], 5)
    k = normed(gen(5), 4, 2, 256)
    k[0, 0, 3], k[0, 0, 40], k[0, 1, 5] = math.inf, -math.inf, math.nan
    k[1] = 0
    k[2] = 1e-4
    cache.write(k, k, [4], [0])
    no_error()
    got = cache.rows(cache.k, 0, 0, 4, 1.0)
    assert float(got[0, 0, 3]) == 2688 and float(got[0, 0, 40]) == -2688 and float(got[0, 1, 5]) == 2688
    assert torch.equal(got[0, 0, 64:], quantised(k[0, 0, 64:], 1.0))
    assert bool((got[1:3] == 0).all()) and torch.equal(got[3], quantised(k[3], 1.0))


def test_write_bad_pages_and_offsets():
    """A bad block id, a position beyond the row, a negative past and rows beyond the host's count are
    left out and flagged; the others are written."""
    layer, g = L256, gen(6)
    for change, bits in (("block", binding.DEVERR_BLOCK_ID), ("row", binding.DEVERR_CAPACITY), ("past", binding.DEVERR_LENGTH),
                         ("count", binding.DEVERR_LENGTH)):
        cache, k = Cache(layer, [40, 40], 7), normed(g, 70, 2, 256)
        past, offsets = [0, 10], cu([40, 30])
        if change == "block":
            cache.table[0, 1] = cache.blocks
        if change == "row":
            past[0] = 20
        if change == "past":
            past[0] = -1
        if change == "count":
            offsets = cu([40, 50])
        binding.kv_cache_write_fp4(layer, k, k, offsets, i32(past), cache.pages, cache.k, cache.v)
        takes_error(bits)
        assert torch.equal(cache.rows(cache.k, 1, 10, 40, 1.0), quantised(k[40:], 1.0))
        if change == "block":
            cache.table[0, 1] = cache.table[0, 0]
            assert torch.equal(cache.rows(cache.k, 0, 0, 16, 1.0), quantised(k[:16], 1.0))


def wide_pages(cache, lens, firsts, seed, spare=2):
    """bf16 pools and a table for the pages of positions [first, len)."""
    layer, n = cache.layer, sum(-(-x // PAGE) - f // PAGE for x, f in zip(lens, firsts)) + spare
    ids = torch.randperm(n, generator=gen(seed), device="cuda").to(torch.int32)
    table, at = torch.full_like(cache.table, -1), 0
    for b, (x, f) in enumerate(zip(lens, firsts)):
        k = max(0, -(-x // PAGE) - f // PAGE)
        table[b, f // PAGE:f // PAGE + k] = ids[at:at + k]
        at += k
    pool = lambda: torch.full((n, PAGE, layer.n_kv_heads, layer.head_dim), 9.0, dtype=BF16, device="cuda")  # noqa: E731
    return binding.make_pages(table, n), pool(), None if layer.k_eq_v else pool()


@pytest.mark.parametrize("layer,lens,firsts,gs", [
    pytest.param(L256, [1], [0], (1.0, 1.0), id="one-token"),
    pytest.param(L256, [16, 0, 17, 100, 31], [0, 0, 16, 37, 30], (1.0, 1.0), id="ragged"),
    pytest.param(Layer(3, 3, 512), [70, 5], [69, 0], (2.0, 0.37), id="512"),
    pytest.param(KEQV, [40, 300], [0, 131], (0.5, 1.0), id="keqv"),
    pytest.param(L512, [(7 * i) % 90 for i in range(700)], [(7 * i) % 90 // 2 for i in range(700)], (1.0, 1.0), id="700-sequences"),
    pytest.param(Layer(8, 8, 256), [7001, 3, 5555], [11, 0, 1003], (1.0, 0.37), id="many"),
    pytest.param(Layer(4, 4, 512, k_eq_v=True), [333, 20001], [300, 17], (1.0, 1.0), id="many-512-keqv"),
])
def test_read(layer, lens, firsts, gs):
    g = gen(8)
    cache = Cache(layer, lens, 9)
    n = sum(lens)
    cache.write(normed(g, n, layer.n_kv_heads, layer.head_dim), None if layer.k_eq_v else normed(g, n, layer.n_kv_heads, layer.head_dim),
                lens, [0] * len(lens), gs)
    pages, k, v = wide_pages(cache, lens, firsts, 10)
    binding.kv_cache_read_fp4(layer, cache.k, cache.v, cache.pages, i32(firsts), i32(lens), pages, k, v, k_scale=gs[0], v_scale=gs[1])
    no_error()
    for wide, pool, s in ((k, cache.k, gs[0]), (v, cache.v, gs[1])):
        if wide is None:
            continue
        done = torch.zeros(wide.shape[:2], dtype=torch.bool, device="cuda")
        for b, (x, f) in enumerate(zip(lens, firsts)):
            if x <= f:
                continue
            pos = torch.arange(f, x, device="cuda")
            at = pages.table[b].long()[pos // PAGE], pos % PAGE
            done[at] = True
            # one rounding to bf16, after the tensor scale's in fp32
            want = cache.rows(pool, b, f, x, s)
            check(wide[at], want, want.abs() * (2.0 ** -8 if s == 0.37 else 0) * 1.001, f"sequence {b}")
        assert bool((wide[~done] == 9).all())


def test_read_bad_pages():
    layer, lens = L256, [40, 40, 40, 40]
    cache, g = Cache(layer, lens, 11), gen(11)
    k = normed(g, 160, 2, 256)
    cache.write(k, k, lens, [0] * 4)
    pages, kw, vw = wide_pages(cache, lens, [0] * 4, 12)
    cache.table[0, 1] = -5
    pages.table[1, 2] = pages.num_blocks
    binding.kv_cache_read_fp4(layer, cache.k, cache.v, cache.pages, None, i32([40, 40, -1, 100]), pages, kw, vw)
    takes_error(binding.DEVERR_BLOCK_ID | binding.DEVERR_LENGTH | binding.DEVERR_CAPACITY)
    want = quantised(k, 1.0)
    t = pages.table.long()
    assert bool((kw[t[0, 1]] == 0).all()) and torch.equal(kw[t[0, 0]].to(F64), want[:16])
    assert torch.equal(vw[t[1, 1]].to(F64), want[56:72])
    assert bool((kw[t[2]] == 9).all())
    assert torch.equal(kw[t[3, 2], :8].to(F64), want[152:160])


# ---------------------------------------------------------------- decode

def decode(layer, cache, q, lens, gs=(1.0, 1.0), ws=None, stream=None):
    n = q.shape[0]
    out = torch.full((n, layer.n_q_heads, layer.head_dim), math.nan, dtype=BF16, device="cuda")
    lse = torch.full((n, layer.n_q_heads), math.nan, device="cuda")
    ws = binding.alloc_fp4_workspace(layer, n) if ws is None else ws
    binding.attn_decode_paged_fp4(layer, q, cache.k, cache.v, cache.pages, i32(lens), out, lse, ws=ws,
                                  k_scale=gs[0], v_scale=gs[1], stream=stream)
    return out, lse


def filled(layer, lens, seed, gs=(1.0, 1.0), spread=1.0, **kw):
    """A cache of normalised rows (times spread) and queries."""
    g, n = gen(seed), sum(lens)
    cache = Cache(layer, lens, seed, **kw)
    shape = (n, layer.n_kv_heads, layer.head_dim)
    k = normed(g, *shape)
    v = None if layer.k_eq_v else (normed(g, *shape).float() * spread).to(BF16)
    cache.write(k, v, lens, [0] * len(lens), gs)
    return cache, normed(g, len(lens), layer.n_q_heads, layer.head_dim)


def compare(layer, cache, q, lens, got, gs=(1.0, 1.0), zero={}):
    out, lse = got
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        check_decode(out[b], lse[b], decode_ref(layer, cache, q, b, n, gs, zero.get(b, ())), f"sequence {b} of {n}")


EDGES = [1, 0, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 0, 255, 256, 257, 500, 1000, 1]


@pytest.mark.parametrize("layer", [
    pytest.param(Layer(2, 2, 256), id="g1"),
    pytest.param(Layer(16, 8, 256, window=100), id="g2-window"),
    pytest.param(Layer(9, 3, 256, scale=0.0625, softcap=50.0), id="g3-softcap"),
    pytest.param(Layer(8, 1, 256, scale=0.2), id="g8"),
    pytest.param(Layer(22, 2, 256, scale=0.3, window=33), id="g11-window"),
    pytest.param(Layer(16, 1, 256, window=1), id="g16-window-1"),
    pytest.param(Layer(8, 2, 512, scale=0.05), id="512-g4"),
    pytest.param(Layer(24, 3, 512, window=70, softcap=5.0, scale=0.1), id="512-g8-window-softcap"),
    pytest.param(Layer(32, 4, 512, k_eq_v=True), id="512-g8-keqv"),
    pytest.param(Layer(10, 1, 512, k_eq_v=True, window=47, scale=0.3), id="512-g10-keqv-window"),
    pytest.param(Layer(6, 2, 256, k_eq_v=True, softcap=30.0), id="256-keqv-softcap"),
])
def test_decode_edges(layer):
    cache, q = filled(layer, EDGES, 20)
    got = decode(layer, cache, q, EDGES)
    no_error()
    compare(layer, cache, q, EDGES, got)


@pytest.mark.parametrize("layer,lens", [
    pytest.param(Layer(4, 2, 256), [20011], id="one-long"),
    pytest.param(Layer(21, 7, 256, scale=0.0625, softcap=50.0), [9001, 3, 12345], id="long-and-short"),
    pytest.param(Layer(8, 1, 512, scale=0.04), [16389], id="one-long-512"),
    pytest.param(Layer(32, 4, 512, k_eq_v=True, scale=0.04), [4000, 100, 2222, 1], id="keqv"),
    pytest.param(Layer(16, 8, 256, window=1024), [700 + 61 * i for i in range(37)], id="sliding-37"),
    pytest.param(Layer(3, 1, 256), [1] * 400, id="400-tokens"),
    pytest.param(Layer(8, 4, 256), [40 + i % 50 for i in range(600)], id="600-short"),
    pytest.param(Layer(16, 2, 512, scale=0.05), [16 * (i % 9) for i in range(500)], id="500-short-512"),
    pytest.param(Layer(8, 8, 256), [0] * 40 + [5] + [0] * 500, id="one-of-541"),
])
def test_decode_batches(layer, lens):
    cache, q = filled(layer, lens, 21)
    got = decode(layer, cache, q, lens)
    no_error()
    compare(layer, cache, q, lens, got)


@pytest.mark.parametrize("layer,lens", [
    pytest.param(Layer(3, 1, 256, scale=0.05), [40000], id="256"),
    pytest.param(Layer(8, 1, 256, window=30000), [9, 33000, 40], id="256-window"),
    pytest.param(Layer(16, 1, 256, softcap=20.0), [12001, 30011], id="256-two-chunks"),
    pytest.param(Layer(2, 1, 512, scale=0.04), [33333], id="512"),
    pytest.param(Layer(16, 2, 512, k_eq_v=True, scale=0.04), [20000, 0, 31000], id="512-keqv"),
])
def test_decode_units_of_many_parts(layer, lens):
    """Contexts that dozens of thread blocks share: their parts are joined in two steps."""
    cache, q = filled(layer, lens, 29)
    ws = binding.alloc_fp4_workspace(layer, len(lens))
    got = decode(layer, cache, q, lens, ws=ws)
    no_error()
    compare(layer, cache, q, lens, got)
    for _ in range(5):
        again = decode(layer, cache, q, lens, ws=ws)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert bool((ws[:binding.FP4_COUNTER_BYTES] == 0).all())


@pytest.mark.parametrize("n", [1, 18, 19, 20])
@pytest.mark.parametrize("layer", [Layer(16, 8, 256, window=900), Layer(8, 8, 512, scale=0.04),
                                   Layer(72, 4, 256, k_eq_v=True, scale=0.05)], ids=["256", "512", "256-keqv-chunks"])
def test_decode_as_many_units_as_blocks(layer, n):
    """Short contexts, some empty, with up to and just beyond as many units as thread blocks; then
    the same with one longer context among them."""
    lens = [(97 * i) % 450 for i in range(1, n)] + [431]
    for extra in (0, 2500):
        lens[n // 2] += extra
        cache, q = filled(layer, lens, 30)
        ws = binding.alloc_fp4_workspace(layer, n)
        got = decode(layer, cache, q, lens, ws=ws)
        no_error()
        compare(layer, cache, q, lens, got)
        assert bool((ws[:binding.FP4_COUNTER_BYTES] == 0).all())


@pytest.mark.parametrize("gs", [(0.37, 2.5), (2.0 ** -20, 2.0 ** 20)])
@pytest.mark.parametrize("layer", [L256, L512], ids=["256", "512"])
def test_decode_tensor_scales(layer, gs):
    lens, g = [300, 77], gen(22)
    cache = Cache(layer, lens, 22)
    shape = (377, layer.n_kv_heads, layer.head_dim)
    k, v = ((normed(g, *shape).float() * s).to(BF16) for s in gs)
    cache.write(k, v, lens, [0, 0], gs)
    q = (normed(g, 2, layer.n_q_heads, layer.head_dim).float() / gs[0]).to(BF16)
    got = decode(layer, cache, q, lens, gs)
    no_error()
    compare(layer, cache, q, lens, got, gs)


@pytest.mark.parametrize("layer", [Layer(4, 2, 256), Layer(8, 1, 512), Layer(8, 1, 512, k_eq_v=True)], ids=["256", "512", "keqv"])
def test_decode_growing_scores(layer):
    """Scores that grow along the context by far more than a running maximum may lag behind, heads whose
    queries differ by many powers of two, values whose rows differ by as many."""
    n, g = 1500, gen(23)
    cache = Cache(layer, [n], 23)
    q = normed(g, 1, layer.n_q_heads, layer.head_dim)
    q = (q.float() * 2.0 ** (-4.0 * torch.arange(layer.n_q_heads, device="cuda")[None, :, None])).to(BF16)
    q[:, 1:] = q[:, :1] * 2.0 ** -7
    d = q[0, 0].float()
    ramp = 0.3 * torch.arange(n, device="cuda")[:, None] / d.square().sum()
    k = (0.3 * randn(g, n, layer.n_kv_heads, layer.head_dim) + (ramp * d)[:, None]).to(BF16)
    v = (randn(g, n, layer.n_kv_heads, layer.head_dim) * 2.0 ** torch.randint(-6, 10, (n, 1, 1), device="cuda", generator=g)).to(BF16)
    cache.write(k, None if layer.k_eq_v else v, [n], [0])
    got = decode(layer, cache, q, [n])
    no_error()
    compare(layer, cache, q, [n], got)


def test_decode_nan_stays_in_its_head():
    """A NaN scale in a visible row shows in its KV head's rows of its sequence alone; one in a slot that
    no key has (behind the end, before the window) in none."""
    layer, lens = Layer(4, 2, 256, window=100), [200, 200, 195]
    cache, q = filled(layer, lens, 24)
    t = cache.table.long()
    cache.v[t[1, 11], 1, 8 * 256:] = 0x7F                       # keys 176..191 of sequence 1, head 1
    for pool in (cache.k, cache.v):
        pool[t[2, 12], :, 8 * 256 + 3 * 16:] = 0x7F             # keys 195.. of sequence 2 do not exist
        pool[t[2, 5], :, 8 * 256:8 * 256 + 15 * 16] = 0x7F      # keys 80..94: its window begins at 95
        pool[t[2, 4]] = 0xFF
    out, lse = decode(layer, cache, q, lens)
    no_error()
    assert bool(out[1, 2:].isnan().all()) and bool(out[1, :2].isfinite().all())
    for b in (0, 2):
        check_decode(out[b], lse[b], decode_ref(layer, cache, q, b, lens[b]), "clean")
    ref = tuple(x[:2] for x in decode_ref(layer, cache, q, 1, 200))
    check_decode(out[1, :2], lse[1, :2], ref, "the other head")


def test_decode_queries_without_finite_values():
    """An infinity or NaN in one head's query makes that head's row NaN and no other."""
    layer, lens = Layer(8, 1, 256), [150]
    cache, q = filled(layer, lens, 25)
    q[0, 2, 7], q[0, 5, 100], q[0, 6] = math.nan, math.inf, 0
    out, lse = decode(layer, cache, q, lens)
    no_error()
    assert bool(out[0, 2].isnan().all()) and bool(out[0, 5].isnan().all())
    keep = [0, 1, 3, 4, 6, 7]
    ref = tuple(x[keep] for x in decode_ref(layer, cache, q, 0, 150))
    check_decode(out[0, keep], lse[0, keep], ref, "the others")


@pytest.mark.parametrize("layer", [L256, KEQV], ids=["256", "512-keqv"])
def test_decode_bad_pages(layer):
    """A block id outside the pool reads as zero rows, a length beyond the table row is clamped, a
    negative one gives an empty row; each is flagged and the others are right."""
    lens = [100, 150, 60, 160, 90]
    cache, q = filled(layer, lens, 26)
    cache.table[0, 2], cache.table[1, 9] = cache.blocks, -1
    got = decode(layer, cache, q, [100, 150, -3, 10000, 90])
    takes_error(binding.DEVERR_BLOCK_ID | binding.DEVERR_CAPACITY | binding.DEVERR_LENGTH)
    cache.table[0, 2] = cache.table[1, 9] = cache.table[0, 0]
    compare(layer, cache, q, [100, 150, 0, 160, 90], got, zero={0: range(32, 48), 1: range(144, 150)})


def test_decode_repeats_and_workspace():
    """Repeated calls in one workspace, larger and smaller batches and both layouts in turn: always the
    same bits, and the counters are zero afterwards."""
    a, b = Layer(16, 8, 256, window=300), Layer(8, 1, 512, k_eq_v=True)
    ca, qa = filled(a, [311 * i % 900 for i in range(50)], 27)
    cb, qb = filled(b, [5000, 17], 28)
    la, lb = [311 * i % 900 for i in range(50)], [5000, 17]
    ws = max((binding.alloc_fp4_workspace(a, 50), binding.alloc_fp4_workspace(b, 2)), key=lambda w: w.numel())
    want_a, want_b = decode(a, ca, qa, la), decode(b, cb, qb, lb)
    for _ in range(3):
        for want, got in ((want_a, decode(a, ca, qa, la, ws=ws)), (want_b, decode(b, cb, qb, lb, ws=ws))):
            assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    no_error()
    assert bool((ws[:binding.FP4_COUNTER_BYTES] == 0).all())


def test_decode_without_lse():
    layer, lens = L512, [700, 3]
    cache, q = filled(layer, lens, 29)
    out, _ = decode(layer, cache, q, lens)
    other = torch.empty_like(out)
    binding.attn_decode_paged_fp4(layer, q, cache.k, cache.v, cache.pages, i32(lens), other, ws=binding.alloc_fp4_workspace(layer, 2))
    no_error()
    assert torch.equal(out, other)


# ---------------------------------------------------------------- tables

def plain_tables(table, past, new, free, at, n_slots):
    table, slots, lens, offsets = [list(r) for r in table], [], [], [0]
    for b, (p, n) in enumerate(zip(past, new)):
        for pos in range(p, p + n):
            page = pos // PAGE
            if pos % PAGE == 0 and page < len(table[b]):
                table[b][page] = free[at] if at < len(free) else -1
                at += at < len(free)
            slots.append(table[b][page] * PAGE + pos % PAGE if page < len(table[b]) and table[b][page] >= 0 else -1)
        lens.append(p + n)
        offsets.append(offsets[-1] + n)
    return table, slots[:n_slots], lens, offsets, at


@pytest.mark.parametrize("n,past_hi,new_hi", [(1, 0, 1), (1, 40, 5000), (64, 4096, 1), (3, 33, 40), (300, 70, 33), (1024, 50, 3),
                                              (1025, 50, 3), (2500, 20, 2), (7, 0, 0)])
@pytest.mark.parametrize("alias", [False, True], ids=["apart", "cursor-in-place"])
def test_tables(n, past_hi, new_hi, alias):
    g = torch.Generator().manual_seed(n)
    past, new = (torch.randint(0, hi + 1, (n,), generator=g).tolist() for hi in (past_hi, new_hi))
    width = max(-(-(p + m) // PAGE) for p, m in zip(past, new)) + 1
    blocks = sum(-(-(p + m) // PAGE) for p, m in zip(past, new)) + 10
    ids = torch.randperm(blocks, generator=g).tolist()
    table, at = [[-1] * width for _ in range(n)], 0
    for b, p in enumerate(past):
        for j in range(-(-p // PAGE)):
            table[b][j] = ids[at]
            at += 1
    free = [-7, -7] + ids[at:]
    rows = sum(new)
    dt, pos, slots = i32(table), i32([2]), torch.full((rows + 3,), -9, dtype=torch.int64, device="cuda")
    nxt = pos if alias else i32([0])
    offsets, lens = i32([5] * (n + 1)), i32([5] * n)
    binding.block_table_extend(dt, i32(past), i32(new), i32(free), pos, nxt, offsets, lens, slots)
    no_error()
    t, s, ln, of, end = plain_tables(table, past, new, free, 2, rows)
    assert dt.tolist() == t and lens.tolist() == ln and offsets.tolist() == of and nxt.tolist() == [end]
    assert slots.tolist() == s + [-9] * 3
    assert alias or pos.tolist() == [2]
    # without slots, and again from the cursor left behind
    dt2, off2, len2 = i32(table), torch.empty_like(offsets), torch.empty_like(lens)
    binding.block_table_extend(dt2, i32(past), i32(new), i32(free), i32([2]), i32([0]), off2, len2)
    no_error()
    assert torch.equal(dt, dt2) and torch.equal(offsets, off2) and torch.equal(lens, len2)


def test_tables_flags():
    """A list that runs out, rows that are too short, bad lengths, few slots, a missing page, a bad cursor."""
    def call(past, new, table, free, at, n_slots):
        dt, nxt, slots = i32(table), i32([0]), torch.full((max(n_slots, 1),), -9, dtype=torch.int64, device="cuda")
        offsets, lens = i32([0] * (len(past) + 1)), i32([0] * len(past))
        binding.block_table_extend(dt, i32(past), i32(new), i32(free), i32([at]), nxt, offsets, lens, slots[:n_slots])
        return dt.tolist(), slots.tolist()[:n_slots], lens.tolist(), offsets.tolist(), int(nxt)

    got = call([0, 10], [40, 10], [[-1] * 3, [5, -1, -1]], [7, 8, 9], 1, 50)
    takes_error(binding.DEVERR_NOBLOCKS)
    assert got[0] == [[8, 9, -1], [5, -1, -1]] and got[4] == 3
    assert got[1] == [8 * 16 + i for i in range(16)] + [9 * 16 + i for i in range(16)] + [-1] * 8 + [5 * 16 + 10 + i for i in range(6)] + [-1] * 4

    got = call([30], [10], [[1, 2]], [3, 4], 0, 10)
    takes_error(binding.DEVERR_CAPACITY)
    assert got == ([[1, 2]], [2 * 16 + 14, 2 * 16 + 15] + [-1] * 8, [40], [0, 10], 0)

    got = call([-5, 3, 4], [2, -1, 1], [[-1], [6], [7]], [3], 0, 1)
    takes_error(binding.DEVERR_LENGTH)
    assert got == ([[-1], [6], [7]], [7 * 16 + 4], [0, 3, 5], [0, 0, 0, 1], 0)

    got = call([0], [5], [[-1]], [3], 0, 2)
    takes_error(binding.DEVERR_LENGTH)
    assert got == ([[3]], [48, 49], [5], [0, 5], 1)

    got = call([5], [1], [[-1]], [3], 0, 1)
    takes_error(binding.DEVERR_BLOCK_ID)
    assert got[1] == [-1]

    for bad in (-1, 4):
        got = call([0], [1], [[9]], [3, 4, 5], bad, 1)
        takes_error(binding.DEVERR_LENGTH | binding.DEVERR_NOBLOCKS)
        assert got == ([[-1]], [-1], [1], [0, 1], 3)

    got = call([2 ** 31 - 20], [100], [[9]], [3], 0, 1)
    takes_error(binding.DEVERR_LENGTH | binding.DEVERR_CAPACITY)
    assert got[3] == [0, 0]


# ---------------------------------------------------------------- together

class Server:
    """As a server runs them: tables, write, read-back and the chunk's prefill, then decode steps."""

    def __init__(self, layer, new, seed, steps=20):
        g = gen(seed)
        self.layer, self.n, self.new = layer, len(new), i32(new)
        total = [x + steps for x in new]
        self.width = max(-(-x // PAGE) for x in total)
        blocks = sum(-(-x // PAGE) for x in total) + 5
        self.free = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        self.cache = Cache(layer, [0] * self.n, seed, spare=blocks, width=self.width)
        self.past, self.lens, self.cur = i32([0] * self.n), i32([0] * self.n), i32([0])
        self.one, self.cu = i32([1] * self.n), i32([0] * (self.n + 1))
        self.ws = binding.alloc_fp4_workspace(layer, self.n)
        self.wide_table = torch.arange(self.n * self.width, dtype=torch.int32, device="cuda").view(self.n, -1)
        self.wide = binding.make_pages(self.wide_table, self.n * self.width)
        self.kw = torch.zeros(self.n * self.width, PAGE, layer.n_kv_heads, layer.head_dim, dtype=BF16, device="cuda")
        self.vw = None if layer.k_eq_v else torch.zeros_like(self.kw)
        row = lambda m: torch.zeros(m, layer.n_kv_heads, layer.head_dim, dtype=BF16, device="cuda")  # noqa: E731
        self.k, self.v = row(self.n), row(self.n)
        self.q = torch.zeros(self.n, layer.n_q_heads, layer.head_dim, dtype=BF16, device="cuda")
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(self.n, layer.n_q_heads, device="cuda")

    def chunk(self, k, v, q):
        layer, c = self.layer, self.cache
        binding.block_table_extend(c.table, self.past, self.new, self.free, self.cur, self.cur, self.cu, self.lens)
        binding.kv_cache_write_fp4(layer, k, v, self.cu, self.past, c.pages, c.k, c.v)
        binding.kv_cache_read_fp4(layer, c.k, c.v, c.pages, None, self.lens, self.wide, self.kw, self.vw)
        out = torch.zeros(q.shape, device="cuda")
        most = int(self.new.max())
        binding.attn_prefill_chunked(layer, q, self.cu, self.past, most, self.kw, self.vw, self.wide, out,
                                     ws=binding.alloc_workspace(layer, self.n, most))
        self.past.copy_(self.lens)
        return out

    def step(self, stream=None):
        layer, c = self.layer, self.cache
        v = None if layer.k_eq_v else self.v
        binding.block_table_extend(c.table, self.past, self.one, self.free, self.cur, self.cur, self.cu, self.lens, stream=stream)
        binding.kv_cache_write_fp4(layer, self.k, v, self.cu, self.past, c.pages, c.k, c.v, stream=stream)
        binding.attn_decode_paged_fp4(layer, self.q, c.k, c.v, c.pages, self.lens, self.out, self.lse, ws=self.ws, stream=stream)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
            self.past.copy_(self.lens)


@pytest.mark.parametrize("layer", [Layer(8, 4, 256, window=64, scale=0.0625, softcap=50.0), Layer(16, 2, 512, k_eq_v=True, scale=0.05)], ids=["sliding", "keqv"])
def test_chain(layer):
    new, g = [70, 5, 33], gen(31)
    s = Server(layer, new, 31)
    T = sum(new)
    k, v = normed(g, T, layer.n_kv_heads, layer.head_dim), normed(g, T, layer.n_kv_heads, layer.head_dim)
    q = normed(g, T, layer.n_q_heads, layer.head_dim)
    out = s.chunk(k, None if layer.k_eq_v else v, q)
    no_error()
    t = 0
    for b, n in enumerate(new):  # the last row of the chunk sees what a decode of it would
        ref = decode_ref(layer, s.cache, q[t + n - 1:t + n].expand(b + 1, -1, -1), b, n)
        # (the prefill's bar: its fp32 result against the pages' rows)
        check(out[t + n - 1], ref[0], 2e-3 + 1e-2 * ref[0].abs(), "chunk")
        t += n
    graph = torch.cuda.CUDAGraph()
    for step in range(20):
        fill = [normed(g, *x.shape) for x in (s.k, s.v, s.q)]
        for dst, src in zip((s.k, s.v, s.q), fill):
            dst.copy_(src)
        if step == 1:
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                s.step()
        if step == 0:
            s.step()
        else:
            graph.replay()
        no_error()
        lens = [n + step + 1 for n in new]
        assert s.lens.tolist() == lens
        compare(layer, s.cache, s.q, lens, (s.out, s.lse))
        for b, n in enumerate(lens):
            assert torch.equal(s.cache.rows(s.cache.k, b, n - 1, n, 1.0)[0], quantised(s.k[b], 1.0))


def test_two_streams():
    """Two steps at once on two streams, each with its own buffers: the bits of one after the other."""
    layer, g = Layer(8, 4, 256), gen(32)
    states = [Server(layer, [900, 40], 33), Server(layer, [333, 1200], 34)]
    want = []
    for s, new in zip(states, ([900, 40], [333, 1200])):
        T = sum(new)
        s.chunk(normed(g, T, 4, 256), normed(g, T, 4, 256), normed(g, T, 8, 256))
        for x in (s.k, s.v, s.q):
            x.copy_(normed(g, *x.shape))
        s.saved = [x.clone() for x in (s.cache.table, s.past, s.cur, s.cache.k, s.cache.v)]
        s.step()
        torch.cuda.synchronize()
        want.append([x.clone() for x in (s.out, s.lse, s.cache.k, s.cache.v, s.cache.table, s.lens)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for s in states:
            for x, y in zip((s.cache.table, s.past, s.cur, s.cache.k, s.cache.v), s.saved):
                x.copy_(y)
            s.out.zero_()
        torch.cuda.synchronize()
        for s, st in zip(states, streams):
            s.step(st)
        torch.cuda.synchronize()
        no_error()
        for s, w in zip(states, want):
            assert all(torch.equal(x, y) for x, y in zip((s.out, s.lse, s.cache.k, s.cache.v, s.cache.table, s.lens), w))


@pytest.mark.parametrize("hd", [256, 512])
def test_far_pages(hd):
    """Pages whose bytes lie beyond 2^31: the bits of the same work on a small pool."""
    layer, g, lens = Layer(6, 3, hd, scale=0.1), gen(35), [70, 200]
    far = 2 ** 31 // (3 * 9 * hd) + 1
    ids = torch.randperm(20, generator=g, device="cuda").to(torch.int32)[:18]
    k, v, q = normed(g, 270, 3, hd), normed(g, 270, 3, hd), normed(g, 2, 6, hd)
    got = []
    for first, blocks in ((0, 20), (far, far + 20)):
        cache = Cache(layer, [0, 0], 1, spare=1, width=13)
        cache.table[0, :5], cache.table[1, :13] = ids[:5] + first, ids[5:18] + first
        cache.blocks, cache.pages = blocks, binding.make_pages(cache.table, blocks)
        cache.k, cache.v = binding.alloc_fp4_pool(layer, blocks), binding.alloc_fp4_pool(layer, blocks)
        cache.write(k, v, lens, [0, 0])
        pages, kw, vw = wide_pages(cache, lens, [0, 0], 36)
        binding.kv_cache_read_fp4(layer, cache.k, cache.v, cache.pages, None, i32(lens), pages, kw, vw)
        got.append((*decode(layer, cache, q, lens), kw, vw))
        no_error()
        del cache
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- refusals of the binding

def test_refusals_of_tensors():
    layer, lens = L256, [30, 20]
    cache, q = filled(layer, lens, 37)
    out, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    ws = binding.alloc_fp4_workspace(layer, 2)
    good = dict(q=q, k=cache.k, v=cache.v, pages=cache.pages, lens=i32(lens), out=out, lse=lse, ws=ws)

    def call(**kw):
        a = {**good, **kw}
        binding.attn_decode_paged_fp4(layer, a["q"], a["k"], a["v"], a["pages"], a["lens"], a["out"], a["lse"], ws=a["ws"])
    call()
    for kw in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q.transpose(1, 2)), dict(k=cache.k[:, :, :100]), dict(k=cache.k.to(torch.int8)),
               dict(out=out.float()), dict(lse=lse.double()), dict(lens=i32(lens).long()), dict(lens=i32(lens).cpu()), dict(ws=ws.cpu()),
               dict(pages=binding.make_pages(cache.table[:1], cache.blocks))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(v=None), dict(ws=None), dict(ws=ws[:1000])):
        with pytest.raises(binding.PswError):
            call(**kw)
    with pytest.raises(binding.PswError):
        binding.attn_decode_paged_fp4(layer, q, cache.k, cache.v, cache.pages, i32(lens), out, ws=ws, k_scale=0.0)
    with pytest.raises(ValueError):
        binding.kv_cache_write_fp4(layer, q[:, :2, :100], q[:, :2], cu([1, 1]), i32([0, 0]), cache.pages, cache.k, cache.v)
    with pytest.raises(ValueError):
        binding.block_table_extend(cache.table, i32([0] * 3), i32([1] * 3), i32([1]), i32([0]), i32([0]), i32([0] * 4), i32([0] * 3))
    no_error()
