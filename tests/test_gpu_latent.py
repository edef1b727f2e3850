"""Latent attention on the GPU against plain 64-bit implementations: cache
write, absorbed decode, expansion, expanded prefill, and the chain of them."""
import math

import pytest
import torch

from latent_harness import (BF16, F64, H_BF16, H_E4M3, NOPE, PAGE, R, THETA, EPS, V, LatentLayer,
                            Pages, attend, check, check_attention, cu, gen, i32, no_error, randn,
                            rot_mag, rotated, row_of, takes_error)
from paged_sliding_window_gb300 import binding

pytestmark = pytest.mark.gpu

# error of a score relative to sum |scale q_d k_d|: fp32 accumulation of up to 576 products, at most
# 2^-23 of the running sum for each of the 36 steps of 16 (tensor core) or 2^-24 for each product
S_ERR = 2.0 ** -17
# FP8 pages: the query enters as three E4M3 parts, each leaving at most 2^-4 of the part before
S_ERR8 = S_ERR + 2.0 ** -12 + 2.0 ** -13
# P enters the product as two bf16 parts (2^-17), or on FP8 pages as three E4M3 parts (2^-12 of P,
# and 2^-19 of the largest P where a part is subnormal)
P_ERR, P_ERR8 = 2.0 ** -16, 2.0 ** -11
# the expanded form rounds P to bf16 once
P_ERR_PREFILL = H_BF16


# ---------------------------------------------------------------- cache write

def _write(L, H, new, past, fp8, weight=True, stride=0, q=True, in_place=False, seed=1):
    g, lens = gen(seed), [n + p for n, p in zip(new, past)]
    pg, T = Pages(lens, L, fp8, seed), sum(new)
    ckv = (3 * randn(g, T + 2, L + R + stride)).to(BF16)[:T, :L + R]
    w = 1 + 0.2 * randn(g, L) if weight else None
    qs = randn(g, T, H, NOPE + R).to(BF16)
    before = qs.clone()
    if in_place:
        q_in = q_out = qs[..., NOPE:]
    else:
        q_in, q_out = qs[..., NOPE:], torch.full((T, H, L + R), 7.0, dtype=BF16, device="cuda")[..., L:]
    if not q:
        q_in = q_out = None
    norm = binding.make_latent_norm(THETA, EPS, w)
    layer = LatentLayer(H, L)
    args = (layer, norm, ckv, q_in, cu(new), i32(past), pg.pages, q_out, pg.pool)
    if fp8:
        binding.latent_norm_rope_cache_write_fp8(*args, pg.scale)
    else:
        binding.latent_norm_rope_cache_write(*args)
    no_error()
    t = 0
    written = torch.zeros(pg.blocks * PAGE, dtype=torch.bool, device="cuda")
    for b, (n, p) in enumerate(zip(new, past)):
        if n == 0:
            continue
        pos = torch.arange(p, p + n, device="cuda")
        want, at = row_of(ckv[t:t + n], pos, L, w), pg.slots(b, p, p + n)
        written[at] = True
        # fp32: the norm is good to a few steps (2^-21), cos and sin to 2^-22
        slop = 2.0 ** -20 * torch.cat([want[:, :L].abs(), rot_mag(ckv[t:t + n, L:])], 1)
        if fp8:
            sc = pg.scale.view(-1)[at].to(F64)
            amax = want.abs().amax(1)
            check(sc, amax / 448, 2.0 ** -18 * amax / 448, "scale")
            got = pg.pool.view(-1, L + R)[at].view(torch.float8_e4m3fn).to(F64) * sc[:, None]
            # half a step of the code: 2^-4 of the value, 2^-10 of the scale where subnormal
            check(got, want, H_E4M3 * want.abs() + 2.0 ** -10 * sc[:, None] + 2 * slop + 2.0 ** -18 * want.abs(), "codes")
        else:
            check(pg.pool.view(-1, L + R)[at], want, H_BF16 * want.abs() + slop, "rows")
        if q:
            src = before[t:t + n, :, NOPE:]
            check(q_out[t:t + n], rotated(src, pos), H_BF16 * rotated(src, pos).abs() + 2.0 ** -20 * rot_mag(src), "queries")
        t += n
    rest = pg.pool.view(-1, L + R)[~written]
    assert bool((rest == 0x7F).all() if fp8 else torch.isnan(rest).all()), "a slot was written that belongs to nobody"
    if in_place:
        assert torch.equal(qs[..., :NOPE], before[..., :NOPE])


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("L,H,new,past,kw", [
    pytest.param(512, 16, [1] * 64, list(range(500, 564)), {}, id="decode64"),
    pytest.param(512, 16, [130, 0, 1, 17], [0, 9, 15, 4095], {}, id="ragged"),
    pytest.param(256, 1, [1], [0], {}, id="one-token-one-head"),
    pytest.param(256, 9, [33, 2], [16777200, 100], dict(stride=8), id="past-2^24-strided"),
    pytest.param(512, 128, [3, 5], [7, 0], dict(weight=False), id="128-heads-weightless"),
    pytest.param(512, 5, [40], [60000], dict(in_place=True), id="in-place"),
    pytest.param(256, 4, [21], [3], dict(q=False), id="cache-only"),
    pytest.param(512, 2, [0, 1] * 600, [5] * 1200, {}, id="1200-sequences"),
    # more than 9728 units: sixteen heads to a warp, the last unit of a token short
    pytest.param(256, 20, [2500, 1, 700], [3, 90, 16], dict(stride=8), id="many-units"),
    pytest.param(512, 33, [1700], [0], dict(in_place=True), id="many-units-in-place"),
])
def test_write(L, H, new, past, kw, fp8):
    if past[0] > 1 << 20:  # a table for far positions would be a gigabyte: share one page
        _write_far(L, H, new, past, fp8)
    else:
        _write(L, H, new, past, fp8, **kw)


def _write_far(L, H, new, past, fp8):
    """Rotation at positions on both sides of 2^24, queries and rows; the pages of the far
    positions are one page, so only the last writer of a slot is compared."""
    g, T = gen(3), sum(new)
    ckv, qs = randn(g, T, L + R + 8).to(BF16)[:, :L + R], randn(g, T, H, R).to(BF16)
    wide = (max(past) + max(new)) // PAGE + 1
    table = torch.zeros(len(new), wide, dtype=torch.int32, device="cuda")
    table[1] = 1
    pool = torch.zeros(2, PAGE, L + R, dtype=torch.uint8 if fp8 else BF16, device="cuda")
    pages, out = binding.make_pages(table, 2), torch.empty_like(qs)
    args = (LatentLayer(H, L), binding.make_latent_norm(THETA, EPS), ckv, qs, cu(new), i32(past), pages, out, pool)
    if fp8:
        binding.latent_norm_rope_cache_write_fp8(*args, torch.zeros(2, PAGE, device="cuda"))
    else:
        binding.latent_norm_rope_cache_write(*args)
    no_error()
    pos = torch.cat([torch.arange(p, p + n, device="cuda") for n, p in zip(new, past)])
    want = rotated(qs, pos)
    check(out, want, H_BF16 * want.abs() + 2.0 ** -20 * rot_mag(qs), "queries")
    if not fp8:
        row = row_of(ckv, pos, L, None)[new[0]:]
        got = pool.view(-1, L + R)[PAGE:][(pos[new[0]:] % PAGE)]
        check(got, row, H_BF16 * row.abs() + 2.0 ** -20 * torch.cat([row[:, :L].abs(), rot_mag(ckv[new[0]:, L:])], 1), "rows")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_write_zero_row(fp8):
    """An all-zero token is a zero row (FP8: scale 0)."""
    pg = Pages([2], 256, fp8, 1)
    ckv = torch.zeros(2, 256 + R, dtype=BF16, device="cuda")
    args = (LatentLayer(1, 256), binding.make_latent_norm(THETA, EPS), ckv, None, cu([2]), i32([0]), pg.pages, None, pg.pool)
    if fp8:
        binding.latent_norm_rope_cache_write_fp8(*args, pg.scale)
        assert bool((pg.scale.view(-1)[pg.slots(0, 0, 2)] == 0).all())
    else:
        binding.latent_norm_rope_cache_write(*args)
    no_error()
    assert bool((pg.rows(0, 0, 2) == 0).all())


def test_write_bad_pages():
    """A block id outside the pool, a position beyond the table row and a negative past are
    flagged and write nothing; their queries are rotated where the position is known."""
    L, H, new, past = 256, 3, [1, 1, 1, 1], [4, 4, 40, -3]
    pg = Pages([16, 16, 16, 16], L, False, 2)
    pg.table[1, 0] = pg.blocks
    ckv, qs = randn(gen(1), 4, L + R).to(BF16), randn(gen(2), 4, H, R).to(BF16)
    out = torch.full_like(qs, 5.0)
    binding.latent_norm_rope_cache_write(LatentLayer(H, L), binding.make_latent_norm(), ckv, qs, cu(new), i32(past), pg.pages, out, pg.pool)
    takes_error(binding.DEVERR_BLOCK_ID | binding.DEVERR_CAPACITY | binding.DEVERR_LENGTH)
    assert int((~torch.isnan(pg.pool.float()).all(-1)).sum()) == 1  # sequence 0's row alone
    pos = torch.tensor([4, 4, 40], device="cuda")
    check(out[:3], rotated(qs[:3], pos), H_BF16 * rotated(qs[:3], pos).abs() + 2.0 ** -20 * rot_mag(qs[:3]), "queries")
    assert bool((out[3] == 5).all())


def test_write_offsets_beyond_the_rows():
    """Offsets that name more rows than there are: the rows there are get written, the rest is
    flagged."""
    L, H = 256, 2
    pg = Pages([64], L, False, 2)
    ckv, qs = randn(gen(1), 20, L + R).to(BF16), randn(gen(2), 20, H, R).to(BF16)
    out = torch.empty_like(qs)
    binding.latent_norm_rope_cache_write(LatentLayer(H, L), binding.make_latent_norm(THETA, EPS), ckv, qs, cu([30]), i32([0]), pg.pages, out, pg.pool)
    takes_error(binding.DEVERR_LENGTH)
    pos = torch.arange(20, device="cuda")
    want = row_of(ckv, pos, L, None)
    slop = 2.0 ** -20 * torch.cat([want[:, :L].abs(), rot_mag(ckv[:, L:])], 1)
    check(pg.pool.view(-1, L + R)[pg.slots(0, 0, 20)], want, H_BF16 * want.abs() + slop, "rows")
    check(out, rotated(qs, pos), H_BF16 * rotated(qs, pos).abs() + 2.0 ** -20 * rot_mag(qs), "queries")
    assert int((~torch.isnan(pg.pool.float()).all(-1)).sum()) == 20


def test_refusals_of_tensors():
    """Shapes, types and tables that would be read out of bounds are refused before the launch."""
    layer, pg = LatentLayer(4, 256), Pages([40, 40], 256, False, 1)
    q, lens = torch.zeros(2, 4, 256 + R, dtype=BF16, device="cuda"), i32([40, 40])
    out, ws = torch.zeros(2, 4, 256, dtype=BF16, device="cuda"), binding.alloc_latent_workspace(layer, 2)
    ok = dict(layer=layer, q=q, pool=pg.pool, pages=pg.pages, seq_lens=lens, out=out, ws=ws)
    binding.attn_decode_latent(**ok)
    for bad in (dict(q=q[:1]), dict(q=q.float()), dict(q=q.cpu()), dict(q=q.transpose(0, 1)), dict(out=out[..., :128]),
                dict(pool=pg.pool[1:]), dict(lse=torch.zeros(2, 3, device="cuda")), dict(seq_lens=lens.long()),
                dict(pages=binding.make_pages(pg.table[:1].contiguous(), pg.blocks))):
        with pytest.raises(ValueError):
            binding.attn_decode_latent(**{**ok, **bad})
    with pytest.raises(binding.PswError) as e:
        binding.attn_decode_latent(**{**ok, "ws": ws[:1024]})
    assert binding.ERRORS[e.value.code] == "PSW_EWORKSPACE"
    w = torch.zeros(4, 256, 256, dtype=BF16, device="cuda")
    kv, rope = torch.zeros(80, 4, 256, dtype=BF16, device="cuda"), torch.zeros(80, R, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        binding.latent_kv_expand(layer, pg.pool, pg.pages, cu([40, 40]), w, kv, rope[:79])
    with pytest.raises(ValueError):
        binding.attn_prefill_latent(layer, torch.zeros(3, 4, 192, dtype=BF16, device="cuda"), cu([3]), i32([0]), 3, kv, rope,
                                    cu([80]), torch.zeros(3, 4, 192, dtype=BF16, device="cuda"))
    no_error()


# ---------------------------------------------------------------- absorbed decode

def _decode_inputs(layer, lens, fp8, seed, q_std=1.0, grow=0.0):
    g, L, H = gen(seed), layer.latent_dim, layer.n_heads
    pg = Pages(lens, L, fp8, seed)
    q = (q_std * randn(g, len(lens), H, L + R)).to(BF16)
    for b, n in enumerate(lens):
        rows = randn(g, n, L + R)
        if grow:  # keys along the first head's query, ever longer
            d = q[b, 0].float()
            rows = 0.1 * rows + d * (grow * torch.arange(n, device="cuda")[:, None] / d.square().sum())
        pg.put(b, rows)
    return pg, q


def _decode_call(layer, pg, q, lens_t, out, lse, ws, stream=None):
    if pg.fp8:
        binding.attn_decode_latent_fp8(layer, q, pg.pool, pg.scale, pg.pages, lens_t, out, lse, ws=ws, stream=stream)
    else:
        binding.attn_decode_latent(layer, q, pg.pool, pg.pages, lens_t, out, lse, ws=ws, stream=stream)


def _decode_ref(layer, pg, q, b, n):
    k = pg.rows(b, 0, n)
    return attend(q[b].to(F64)[:, None], k[None], k[None, :, :layer.latent_dim],
                  torch.tensor([n - 1], device="cuda"), torch.arange(n, device="cuda"), layer)


def _run_decode(layer, lens, fp8, seed=5, **kw):
    pg, q = _decode_inputs(layer, lens, fp8, seed, **kw)
    n, H, L = len(lens), layer.n_heads, layer.latent_dim
    out = torch.full((n, H, L), float("nan"), dtype=BF16, device="cuda")
    lse = torch.full((n, H), float("nan"), device="cuda")
    ws = binding.alloc_latent_workspace(layer, n)
    ws.fill_(0xFF)
    _decode_call(layer, pg, q, i32(lens), out, lse, ws)
    no_error()
    for b, ln in enumerate(lens):
        if ln == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        o, l, a, m = _decode_ref(layer, pg, q, b, ln)
        check_attention(out[b][:, None], lse[b][:, None], (o, l, a, m), P_ERR8 if fp8 else P_ERR,
                        S_ERR8 if fp8 else S_ERR, f"sequence {b} of {ln}")
    return out, lse


EDGES = [1, 0, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 144, 255, 256, 257, 0, 500, 1000, 1]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("layer", [
    pytest.param(LatentLayer(16, 512, scale=0.07), id="L512-h16"),
    pytest.param(LatentLayer(1, 256, scale=0.07), id="L256-h1"),
    pytest.param(LatentLayer(17, 256, scale=0.07, window=40), id="L256-h17-w40"),
    pytest.param(LatentLayer(32, 512, scale=0.07, softcap=30.0), id="L512-h32-cap"),
    pytest.param(LatentLayer(33, 512, scale=0.07, window=128), id="L512-h33-w128"),
    pytest.param(LatentLayer(128, 512, scale=0.07, window=1), id="L512-h128-w1"),
    pytest.param(LatentLayer(24, 256, scale=0.3, softcap=2.0, window=300), id="L256-h24-w300-cap2"),
    pytest.param(LatentLayer(64, 512, scale=0.07), id="L512-h64"),
])
def test_decode_edges(layer, fp8):
    _run_decode(layer, EDGES, fp8)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("lens,heads", [([20011], 16), ([9001, 3], 40), ([700] * 37, 8), ([1] * 400, 3)],
                         ids=["one-long", "long-and-short", "37x700", "400x1"])
def test_decode_batches(lens, heads, fp8):
    """One sequence over every SM, unequal ones, more units than SMs."""
    _run_decode(LatentLayer(heads, 512, scale=0.07), lens, fp8)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_growing_scores(fp8):
    """Scores that grow along the context by far more than a running maximum may lag behind."""
    layer = LatentLayer(4, 256, scale=1.0)
    _run_decode(layer, [1500, 300], fp8, grow=2.0)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_peaked_and_flat(fp8):
    _run_decode(LatentLayer(16, 512, scale=1.0), [3000, 129], fp8, q_std=1.0)
    _run_decode(LatentLayer(16, 512, scale=1e-4), [3000, 129], fp8)


def test_decode_uneven_row_scales():
    """FP8 rows whose scales differ by a factor of a million, zero rows among them."""
    layer = LatentLayer(8, 512, scale=0.05)
    lens = [700, 40]
    pg, q = _decode_inputs(layer, lens, True, 8)
    g = gen(4)
    for b, n in enumerate(lens):
        rows = randn(g, n, 512 + R) * 10.0 ** (-6 * torch.rand(n, 1, generator=g, device="cuda"))
        rows[::7] = 0
        pg.put(b, rows)
    out, lse = torch.empty(2, 8, 512, dtype=BF16, device="cuda"), torch.empty(2, 8, device="cuda")
    _decode_call(layer, pg, q, i32(lens), out, lse, binding.alloc_latent_workspace(layer, 2))
    no_error()
    for b, n in enumerate(lens):
        check_attention(out[b][:, None], lse[b][:, None], _decode_ref(layer, pg, q, b, n), P_ERR8, S_ERR8, "uneven")


def test_decode_nan_in_visible_key_stays_in_its_sequence():
    layer = LatentLayer(4, 256, scale=0.07)
    lens = [200, 200, 200]
    pg, q = _decode_inputs(layer, lens, False, 9)
    pg.pool.view(-1, 256 + R)[pg.slots(1, 77, 78)] = float("nan")
    out, lse = torch.empty(3, 4, 256, dtype=BF16, device="cuda"), torch.empty(3, 4, device="cuda")
    _decode_call(layer, pg, q, i32(lens), out, lse, binding.alloc_latent_workspace(layer, 3))
    no_error()
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
    for b in (0, 2):
        check_attention(out[b][:, None], lse[b][:, None], _decode_ref(layer, pg, q, b, 200), P_ERR, S_ERR, "clean")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_bad_pages(fp8):
    """A block id outside the pool reads as zero rows, a length beyond the table row is clamped,
    a negative one gives an empty row; each is flagged and the others are right."""
    layer = LatentLayer(8, 512, scale=0.07)
    lens = [100, 64, 64, 112]
    pg, q = _decode_inputs(layer, lens, fp8, 6)
    full = pg.table.shape[1] * PAGE
    assert full == 112
    bad = int(pg.table[0, 2])
    pg.table[0, 2] = pg.blocks + 5
    ask = i32([100, 64, -5, full + 900])
    out, lse = torch.empty(4, 8, 512, dtype=BF16, device="cuda"), torch.empty(4, 8, device="cuda")
    _decode_call(layer, pg, q, ask, out, lse, binding.alloc_latent_workspace(layer, 4))
    takes_error(binding.DEVERR_BLOCK_ID | binding.DEVERR_CAPACITY | binding.DEVERR_LENGTH)
    p, s = (P_ERR8, S_ERR8) if fp8 else (P_ERR, S_ERR)
    check_attention(out[3][:, None], lse[3][:, None], _decode_ref(layer, pg, q, 3, full), p, s, "clamped")
    assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())
    pg.table[0, 2] = bad
    k = pg.rows(0, 0, 100)
    k[32:48] = 0
    ref = attend(q[0].to(F64)[:, None], k[None], k[None, :, :512], torch.tensor([99], device="cuda"),
                 torch.arange(100, device="cuda"), layer)
    check_attention(out[0][:, None], lse[0][:, None], ref, p, s, "missing page")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_streams_and_graphs(fp8):
    """Two calls at once on two streams with a workspace each, and a captured call replayed on
    new data in the same buffers: the bits of a plain call."""
    layer = LatentLayer(16, 512, scale=0.07)
    lens = [3000, 17, 900]
    one, two = (_decode_inputs(layer, lens, fp8, s) for s in (11, 12))
    lens_t, plain, wss = i32(lens), [], [binding.alloc_latent_workspace(layer, 3) for _ in range(2)]
    for pg, q in (one, two):
        out, lse = torch.empty(3, 16, 512, dtype=BF16, device="cuda"), torch.empty(3, 16, device="cuda")
        _decode_call(layer, pg, q, lens_t, out, lse, wss[0])
        plain.append((out, lse))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for (pg, q), s, ws in zip((one, two), streams, wss):
        out, lse = torch.zeros(3, 16, 512, dtype=BF16, device="cuda"), torch.zeros(3, 16, device="cuda")
        got.append((out, lse))
    torch.cuda.synchronize()
    for rep in range(4):
        for (pg, q), s, ws, (out, lse) in zip((one, two), streams, wss, got):
            _decode_call(layer, pg, q, lens_t, out, lse, ws, stream=s)
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(plain, got):
        assert torch.equal(a, c) and torch.equal(b, d)
    pg, q = one
    q = q.clone()
    out, lse = torch.zeros_like(plain[0][0]), torch.zeros_like(plain[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _decode_call(layer, pg, q, lens_t, out, lse, wss[0])
    q.copy_(two[1])
    pg.pool.copy_(two[0].pool)
    pg.table.copy_(two[0].table)
    if fp8:
        pg.scale.copy_(two[0].scale)
    for _ in range(2):
        graph.replay()
    no_error()
    assert torch.equal(out, plain[1][0]) and torch.equal(lse, plain[1][1])


# ---------------------------------------------------------------- expansion

def _w(g, H, L):
    return (randn(g, H, NOPE + V, L) / math.sqrt(L)).to(BF16)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("L,H,lens,first", [
    pytest.param(512, 16, [130, 0, 1, 17, 128], None, id="ragged"),
    pytest.param(256, 1, [1], None, id="one"),
    pytest.param(256, 3, [700, 65], [0, 33], id="offset"),
    pytest.param(512, 128, [40, 3], [16, 1000], id="128-heads"),
    pytest.param(512, 5, [1] * 300, None, id="300-sequences"),
    pytest.param(256, 1, [26001, 19000], [0, 7], id="several-tiles"),
    pytest.param(512, 1, [40001], None, id="several-tiles-512"),
])
def test_expand(L, H, lens, first, fp8):
    g, first_l = gen(7), first or [0] * len(lens)
    pg = Pages([n + f for n, f in zip(lens, first_l)], L, fp8, 7)
    for b, (n, f) in enumerate(zip(lens, first_l)):
        pg.put(b, randn(g, n + f, L + R))
    w, T = _w(g, H, L), sum(lens)
    kv = torch.full((T + 5, H, NOPE + V), 3.0, dtype=BF16, device="cuda")
    rope = torch.full((T + 5, R), 3.0, dtype=BF16, device="cuda")
    kf = None if first is None else i32(first)
    if fp8:
        binding.latent_kv_expand_fp8(LatentLayer(H, L), pg.pool, pg.scale, pg.pages, cu(lens), w, kv, rope, k_first=kf)
    else:
        binding.latent_kv_expand(LatentLayer(H, L), pg.pool, pg.pages, cu(lens), w, kv, rope, k_first=kf)
    no_error()
    assert bool((kv[T:] == 3).all()) and bool((rope[T:] == 3).all())
    rows = torch.cat([pg.rows(b, f, n + f) for b, (n, f) in enumerate(zip(lens, first_l))])
    wd = w.to(F64)
    want = torch.einsum("tl,hel->the", rows[:, :L], wd)
    mag = torch.einsum("tl,hel->the", rows[:, :L].abs(), wd.abs())
    check(kv[:T], want, H_BF16 * want.abs() + S_ERR * mag, "kv")
    check(rope[:T], rows[:, L:], H_BF16 * rows[:, L:].abs() + 1e-30, "rope")


def test_expand_bad_pages():
    L, H, lens = 256, 2, [40, 40, 40]
    g, pg = gen(1), Pages([40, 40, 40], 256, False, 3)
    for b in range(3):
        pg.put(b, randn(g, 40, L + R))
    pg.table[0, 1] = -7
    w = _w(g, H, L)
    kv, rope = torch.full((120, H, 256), 3.0, dtype=BF16, device="cuda"), torch.full((120, R), 3.0, dtype=BF16, device="cuda")
    binding.latent_kv_expand(LatentLayer(H, L), pg.pool, pg.pages, cu(lens), w, kv, rope, k_first=i32([0, -1, 20]))
    takes_error(binding.DEVERR_BLOCK_ID | binding.DEVERR_CAPACITY | binding.DEVERR_LENGTH)
    assert bool((kv[16:32] == 0).all()) and bool((rope[16:32] == 0).all())
    assert bool((kv[40:80] == 0).all())       # negative first position
    assert bool((kv[108:] == 0).all())        # positions 48.. beyond the row's 3 pages
    keep = torch.cat([pg.rows(0, 0, 16), pg.rows(0, 32, 40)])
    got = torch.cat([kv[:16], kv[32:40]])
    want = torch.einsum("tl,hel->the", keep[:, :L], w.to(F64))
    check(got, want, H_BF16 * want.abs() + S_ERR * torch.einsum("tl,hel->the", keep[:, :L].abs(), w.to(F64).abs()), "others")


# ---------------------------------------------------------------- expanded prefill

def _run_prefill(layer, new, past, first=None, keys=None, seed=21, spare=3, q_std=1.0):
    g, H, n = gen(seed), layer.n_heads, len(new)
    first_l = first or [0] * n
    keys = keys or [p + s - f for p, s, f in zip(past, new, first_l)]
    T, K = sum(new), sum(keys)
    q = (q_std * randn(g, T + spare, H, NOPE + R)).to(BF16)
    kv, rope = randn(g, K + spare, H, NOPE + V).to(BF16), randn(g, K + spare, R).to(BF16)
    kv[K:], rope[K:] = float("nan"), float("nan")
    out = torch.full((T + spare, H, V), 3.0, dtype=BF16, device="cuda")
    lse = torch.full((T + spare, H), 3.0, device="cuda")
    binding.attn_prefill_latent(layer, q, cu(new), i32(past), max(new), kv, rope, cu(keys), out, lse,
                                k_first=None if first is None else i32(first))
    no_error()
    assert bool((out[T:] == 3).all()) and bool((lse[T:] == 3).all()), "rows behind the last sequence"
    q0 = k0 = 0
    for b in range(n):
        if new[b]:
            k = torch.cat([kv[k0:k0 + keys[b], :, :NOPE], rope[k0:k0 + keys[b], None].expand(-1, H, -1)], -1)
            ref = attend(q[q0:q0 + new[b]].to(F64).transpose(0, 1), k.to(F64).transpose(0, 1),
                         kv[k0:k0 + keys[b], :, NOPE:].to(F64).transpose(0, 1),
                         past[b] + torch.arange(new[b], device="cuda"),
                         first_l[b] + torch.arange(keys[b], device="cuda"), layer)
            check_attention(out[q0:q0 + new[b]].transpose(0, 1), lse[q0:q0 + new[b]].transpose(0, 1), ref,
                            P_ERR_PREFILL, S_ERR, f"sequence {b}")
        q0, k0 = q0 + new[b], k0 + keys[b]


@pytest.mark.parametrize("layer,new,past,kw", [
    pytest.param(LatentLayer(4, scale=0.07), [1, 0, 2, 17], [0, 5, 127, 128], {}, id="short"),
    pytest.param(LatentLayer(3, scale=0.07), [128, 129, 255, 256, 257], [0, 1, 127, 128, 300], {}, id="tile-edges"),
    pytest.param(LatentLayer(1, scale=0.07), [700], [1000], {}, id="one-head"),
    pytest.param(LatentLayer(16, scale=0.07, softcap=30.0), [300, 40], [77, 900], {}, id="softcap"),
    pytest.param(LatentLayer(2, scale=0.07, window=100), [300, 513], [777, 0], {}, id="window"),
    pytest.param(LatentLayer(2, scale=0.07, window=1), [260], [50], {}, id="window-1"),
    pytest.param(LatentLayer(5, scale=0.3, window=128, softcap=2.0), [129, 64], [128, 640], {}, id="window-softcap"),
    pytest.param(LatentLayer(2, scale=0.07, window=64), [100, 30], [500, 90], dict(first=[437, 27]), id="first"),
    pytest.param(LatentLayer(2, scale=0.07), [64, 32], [0, 10], dict(first=[40, 0], keys=[20, 42]), id="rows-with-no-key"),
    pytest.param(LatentLayer(2, scale=0.07), [64, 32], [10, 10], dict(keys=[0, 5]), id="few-or-no-keys"),
    pytest.param(LatentLayer(128, scale=0.07), [33], [10], {}, id="128-heads"),
    pytest.param(LatentLayer(2, scale=2.0), [300], [500], {}, id="peaked"),
    pytest.param(LatentLayer(1, scale=0.07), [1] * 300, list(range(300)), {}, id="300-sequences"),
    # short chunks of many heads and sequences, done by single CTAs
    pytest.param(LatentLayer(20, scale=0.07), [128, 129, 255, 256, 1, 0], [0, 1, 95, 96, 300, 7], {}, id="single-edges"),
    pytest.param(LatentLayer(40, scale=0.07, window=70, softcap=4.0), [200, 30], [333, 1], {}, id="single-window-softcap"),
    pytest.param(LatentLayer(40, scale=0.07), [200, 250, 130], [0, 10, 0], dict(first=[140, 0, 0], keys=[50, 260, 0]), id="single-few-or-no-keys"),
    # more pieces than CTAs: those take several, some of them without rows or keys
    pytest.param(LatentLayer(16, scale=0.07), [37 * i % 200 for i in range(40)], [113 * i % 700 for i in range(40)], {}, id="single-many"),
    pytest.param(LatentLayer(8, scale=0.07, window=50), [i % 5 for i in range(300)], [7 * i for i in range(300)],
                 dict(first=[max(0, 7 * i - 60) for i in range(300)]), id="single-many-short"),
    pytest.param(LatentLayer(24, scale=0.07, window=200), [0, 300, 1, 900, 600, 257], [5, 0, 900, 130, 1, 300], {}, id="pair-many"),
    pytest.param(LatentLayer(20, scale=0.07, softcap=20.0), [300, 520, 0, 40, 700, 1], [0, 10, 3, 0, 5, 0],
                 dict(keys=[0, 130, 0, 40, 1, 0]), id="pair-many-few-keys"),
    # keys split between the two halves of a CTA
    pytest.param(LatentLayer(20, scale=0.07), [128, 127, 1, 0, 50], [0, 97, 95, 0, 1000], {}, id="split-edges"),
    pytest.param(LatentLayer(40, scale=0.07, window=200, softcap=4.0), [100, 30], [633, 1], {}, id="split-window-softcap"),
    pytest.param(LatentLayer(40, scale=0.07), [100, 120, 30], [0, 10, 0], dict(first=[60, 0, 0], keys=[30, 130, 0]), id="split-few-or-no-keys"),
    pytest.param(LatentLayer(4, scale=0.07), [256, 1, 129], [0, 128, 383], {}, id="pair-split-edges"),
    pytest.param(LatentLayer(3, scale=0.07, window=300), [200, 256], [1333, 1], {}, id="pair-split-window"),
    # chunks of more than 256 rows, done by pairs of CTAs, 512 rows each
    pytest.param(LatentLayer(3, scale=0.07), [512, 511, 257, 1, 0], [0, 129, 2048, 3000, 7], {}, id="pair-edges"),
    pytest.param(LatentLayer(2, scale=0.07), [1300, 513], [1, 700], {}, id="pair-blocks"),
    pytest.param(LatentLayer(2, scale=0.07, window=90, softcap=4.0), [1025, 260], [300, 1], {}, id="pair-window"),
    pytest.param(LatentLayer(2, scale=0.07), [600, 300], [0, 10], dict(first=[400, 0], keys=[150, 310]), id="pair-rows-with-no-key"),
    pytest.param(LatentLayer(2, scale=0.07), [600, 400, 300], [10, 10, 0], dict(keys=[0, 5, 128]), id="pair-few-or-no-keys"),
    pytest.param(LatentLayer(1, scale=0.07, window=64), [300] + [1] * 299, [500] * 300, dict(first=[400] + [437] * 299), id="pair-300-sequences"),
    pytest.param(LatentLayer(40, scale=0.07), [700, 280, 600], [100, 1500, 0], {}, id="pair-more-work-than-pairs"),
])
def test_prefill(layer, new, past, kw):
    _run_prefill(layer, new, past, **kw)


def test_prefill_no_keys_at_all():
    layer = LatentLayer(2, scale=0.07)
    q = randn(gen(1), 5, 2, NOPE + R).to(BF16)
    out, lse = torch.ones(5, 2, V, dtype=BF16, device="cuda"), torch.ones(5, 2, device="cuda")
    empty = torch.empty(0, 2, NOPE + V, dtype=BF16, device="cuda")
    binding.attn_prefill_latent(layer, q, cu([5]), i32([0]), 5, empty, torch.empty(0, R, dtype=BF16, device="cuda"), cu([0]), out, lse)
    no_error()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("n,t,H", [(200, 900, 2), (700, 1500, 2), (200, 900, 80), (100, 900, 80)])
def test_prefill_growing_scores(n, t, H):
    """Scores that grow along the context by far more than a running maximum may lag behind."""
    layer = LatentLayer(H, scale=1.0)
    g = gen(2)
    q = randn(g, n, H, NOPE + R).to(BF16)
    q[:, :, :] = q[:1, :1]
    d = q[0, 0].float()
    ramp = 1.5 * torch.arange(t, device="cuda")[:, None] / d.square().sum()
    kv = 0.1 * randn(g, t, H, NOPE + V)
    kv[:, :, :NOPE] += (ramp * d[:NOPE])[:, None]
    kv[..., NOPE:] = randn(g, t, H, V)
    kv, rope = kv.to(BF16), (ramp * d[NOPE:]).to(BF16)
    out, lse = torch.empty(n, H, V, dtype=BF16, device="cuda"), torch.empty(n, H, device="cuda")
    binding.attn_prefill_latent(layer, q, cu([n]), i32([t - n]), n, kv, rope, cu([t]), out, lse)
    no_error()
    k = torch.cat([kv[..., :NOPE], rope[:, None].expand(-1, H, -1)], -1)
    ref = attend(q.to(F64).transpose(0, 1), k.to(F64).transpose(0, 1), kv[..., NOPE:].to(F64).transpose(0, 1),
                 t - n + torch.arange(n, device="cuda"), torch.arange(t, device="cuda"), layer)
    check_attention(out.transpose(0, 1), lse.transpose(0, 1), ref, P_ERR_PREFILL, S_ERR, "growing")


def test_prefill_bad_lengths():
    """A chunk longer than max_q_len is cut and flagged, a negative past skips its sequence."""
    layer = LatentLayer(2, scale=0.07)
    g, new, past = gen(1), [20, 10], [0, -1]
    q, kv, rope = randn(g, 30, 2, NOPE + R).to(BF16), randn(g, 30, 2, NOPE + V).to(BF16), randn(g, 30, R).to(BF16)
    out = torch.full((30, 2, V), 3.0, dtype=BF16, device="cuda")
    binding.attn_prefill_latent(layer, q, cu(new), i32(past), 16, kv, rope, cu(new), out)
    takes_error(binding.DEVERR_LENGTH)
    assert bool((out[16:] == 3).all())
    k = torch.cat([kv[:20, :, :NOPE], rope[:20, None].expand(-1, 2, -1)], -1)
    ref = attend(q[:16].to(F64).transpose(0, 1), k.to(F64).transpose(0, 1), kv[:20, :, NOPE:].to(F64).transpose(0, 1),
                 torch.arange(16, device="cuda"), torch.arange(20, device="cuda"), layer)
    check_attention(out[:16].transpose(0, 1), None, ref, P_ERR_PREFILL, S_ERR, "cut")


def test_prefill_stream_and_graph():
    layer, new, past = LatentLayer(4, scale=0.07), [130, 40], [300, 0]
    g = gen(5)
    q, kv, rope = randn(g, 170, 4, NOPE + R).to(BF16), randn(g, 470, 4, NOPE + V).to(BF16), randn(g, 470, R).to(BF16)
    args = (cu(new), i32(past), 130, kv, rope, cu([430, 40]))
    a, b = (torch.zeros(170, 4, V, dtype=BF16, device="cuda") for _ in range(2))
    binding.attn_prefill_latent(layer, q, *args, a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    binding.attn_prefill_latent(layer, q, *args, b, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.attn_prefill_latent(layer, q, *args, b)
    b.zero_()
    graph.replay()
    no_error()
    assert torch.equal(a, b)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_chain_prefill_then_decode(fp8):
    """As a server runs them: chunks written, expanded and attended to; then a decode step whose
    absorbed result, projected by the value weights, is what the expanded form gives that token."""
    L, H, new, past = 512, 4, [150, 33], [0, 0]
    layer = LatentLayer(H, L, scale=1 / math.sqrt(NOPE + R))
    g, total = gen(13), [n + 1 for n in new]
    pg, w = Pages(total, L, fp8, 13), _w(g, H, L)
    norm = binding.make_latent_norm(THETA, EPS, 1 + 0.1 * randn(g, L))

    def write(ckv, q, q_out, lens, before):
        args = (layer, norm, ckv, q, cu(lens), i32(before), pg.pages, q_out, pg.pool)
        if fp8:
            binding.latent_norm_rope_cache_write_fp8(*args, pg.scale)
        else:
            binding.latent_norm_rope_cache_write(*args)

    def expanded(q, lens, before):
        keys = [n + p for n, p in zip(lens, before)]
        kv, rope = torch.empty(sum(keys), H, 256, dtype=BF16, device="cuda"), torch.empty(sum(keys), R, dtype=BF16, device="cuda")
        if fp8:
            binding.latent_kv_expand_fp8(layer, pg.pool, pg.scale, pg.pages, cu(keys), w, kv, rope)
        else:
            binding.latent_kv_expand(layer, pg.pool, pg.pages, cu(keys), w, kv, rope)
        out = torch.empty(q.shape[0], H, V, dtype=BF16, device="cuda")
        binding.attn_prefill_latent(layer, q, cu(lens), i32(before), max(lens), kv, rope, cu(keys), out)
        return out, kv

    def ref(q, b, p):
        """64 bits from the pool's rows and the rotated queries."""
        rows = pg.rows(b, 0, int(p[-1]) + 1)
        kv = torch.einsum("tl,hel->hte", rows[:, :L], w.to(F64))
        k = torch.cat([kv[..., :NOPE], rows[None, :, L:].expand(H, -1, -1)], -1)
        return attend(q.to(F64).transpose(0, 1), k, kv[..., NOPE:], p, torch.arange(rows.shape[0], device="cuda"), layer)

    # the pages' rows are the ones compared with, so the bound counts what follows them: key and
    # value components rounded to bf16 (scores off by 2^-8 of their magnitude at most, twice; values
    # by 2^-8), P to bf16, the result once
    s_err = H_BF16 + S_ERR
    q = randn(g, sum(new), H, NOPE + R).to(BF16)
    write(randn(g, sum(new), L + R).to(BF16), q[..., NOPE:], q[..., NOPE:], new, past)
    out, _ = expanded(q, new, past)
    no_error()
    at = 0
    for b, n in enumerate(new):
        check_attention(out[at:at + n].transpose(0, 1), None, ref(q[at:at + n], b, torch.arange(n, device="cuda")),
                        2 * H_BF16, s_err, "chunk")
        at += n
    # one new token each
    q1 = randn(g, 2, H, NOPE + R).to(BF16)
    q_abs = torch.empty(2, H, L + R, dtype=BF16, device="cuda")
    q_abs[..., :L] = torch.einsum("bhn,hnl->bhl", q1[..., :NOPE].float(), w[:, :NOPE].float()).to(BF16)
    ckv1 = randn(g, 2, L + R).to(BF16)
    write(ckv1, q1[..., NOPE:], q_abs[..., L:], [1, 1], new)
    lat = torch.empty(2, H, L, dtype=BF16, device="cuda")
    _decode_call(layer, pg, q_abs, i32(total), lat, None, binding.alloc_latent_workspace(layer, 2))
    no_error()
    q1[..., NOPE:] = q_abs[..., L:]
    for b in range(2):
        o, l, a, m = ref(q1[b:b + 1], b, torch.tensor([new[b]], device="cuda"))
        # absorbed queries rounded to bf16: their score's magnitude is at most sum |q'||c|
        rows = pg.rows(b, 0, total[b])
        mag = layer.scale * torch.matmul(q_abs[b].to(F64).abs(), rows.abs().t()).amax(-1)[:, None]
        got = torch.einsum("hl,hvl->hv", lat[b].to(F64), w[:, NOPE:].to(F64))[:, None]
        wide = torch.einsum("hl,hvl->hv", lat[b].to(F64).abs(), w[:, NOPE:].to(F64).abs())[:, None]
        e = (mag * H_BF16).clamp(max=0.25)
        check(got, o, H_BF16 * wide * 1.1 + a * (3 * e + (P_ERR8 if fp8 else P_ERR))[..., None] * 1.1 + 1e-30, "decode")
