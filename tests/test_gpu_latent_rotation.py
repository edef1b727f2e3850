"""The latent cache write at far positions, rows and queries, and the rotated queries of the
captured and concurrent chain, on both kinds of pages."""
import pytest
import torch

from latent_harness import (BF16, EPS, F64, H_BF16, H_E4M3, NOPE, PAGE, R, THETA, V, LatentLayer, binding, check, cu, gen,
                            i32, no_error, randn, rot_mag, rotated, row_of)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("first", [16777200, 2 ** 22 - 9, 2 ** 31 - 64, 1 << 29], ids=["2^24", "2^22", "2^31", "2^29"])
def test_far_positions(first, fp8):
    """33 tokens from `first` on, in pages of their own, and 2 of a near sequence: strided rows,
    strided queries."""
    L, H, new, past = 256, 9, [33, 2], [first, 100]
    g, T = gen(3), sum(new)
    ckv = (2 * randn(g, T, L + R + 8)).to(BF16)[:, :L + R]
    buf = randn(g, T, H, NOPE + R + 8).to(BF16)
    qs, out = buf[..., NOPE:NOPE + R], torch.full((T, H, L + R), 7.0, dtype=BF16, device="cuda")[..., L:]
    w = 1 + 0.2 * randn(g, L)
    blocks, wide = 12, (first + new[0] - 1) // PAGE + 1
    table = torch.full((2, wide), -1, dtype=torch.int32, device="cuda")
    pages_used = range(first // PAGE, wide)
    for i, p in enumerate(pages_used):
        table[0, p] = 10 - i
    table[1, 6] = 1
    if fp8:
        pool, scale = torch.full((blocks, PAGE, L + R), 0x7F, dtype=torch.uint8, device="cuda"), torch.full((blocks, PAGE), float("nan"), device="cuda")
    else:
        pool, scale = torch.full((blocks, PAGE, L + R), float("nan"), dtype=BF16, device="cuda"), None
    args = (LatentLayer(H, L), binding.make_latent_norm(THETA, EPS, w), ckv, qs, cu(new), i32(past), binding.make_pages(table, blocks), out, pool)
    if fp8:
        binding.latent_norm_rope_cache_write_fp8(*args, scale)
    else:
        binding.latent_norm_rope_cache_write(*args)
    no_error()
    pos = torch.cat([torch.arange(p, p + n, device="cuda") for n, p in zip(new, past)])
    want = rotated(qs, pos)
    # fp32 sine and cosine (2^-20), and on both sides an angle pos * f in 64 bits: f (1 + 2 |ln f|) <= 1.3
    # half steps of f, half a step of the product, 2^-50 pos for the two together
    err = (2.0 ** -20 + 2.0 ** -50 * pos.to(F64))
    check(out, want, H_BF16 * want.abs() + err[:, None, None] * rot_mag(qs), "queries")
    seq = torch.tensor([0] * new[0] + [1] * new[1], device="cuda")
    slot = table[seq, pos // PAGE].long() * PAGE + pos % PAGE
    row = row_of(ckv, pos, L, w)
    slop = err[:, None] * torch.cat([row[:, :L].abs(), rot_mag(ckv[:, L:])], 1)
    got = pool.view(-1, L + R)[slot]
    if fp8:
        sc, amax = scale.view(-1)[slot].to(F64), row.abs().amax(1)
        check(sc, amax / 448, (2.0 ** -18 * amax + slop.amax(1)) / 448, "scales")
        got = got.view(torch.float8_e4m3fn).to(F64) * sc[:, None]
        check(got, row, H_E4M3 * row.abs() + 2.0 ** -10 * sc[:, None] + 2 * slop + 2.0 ** -18 * row.abs(), "codes")
    else:
        check(got, row, H_BF16 * row.abs() + slop, "rows")
    rest = torch.ones(blocks * PAGE, dtype=torch.bool, device="cuda")
    rest[slot] = False
    left = pool.view(-1, L + R)[rest]
    assert bool((left == 0x7F).all() if fp8 else torch.isnan(left).all())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("H,new", [(4, [150, 33]), (48, [90, 200]), (24, [600, 20])], ids=["spare-pairs", "singles", "pairs"])
def test_chain_rotated_queries(H, new, fp8):
    """Write, expansion, chunk attention over the rotated queries, and decode, captured and
    replayed with other inputs and on two streams at once: the rotated queries and everything
    behind them are what the calls give one by one, on both kinds of pages."""
    L, n = 512, len(new)
    layer, g, T = LatentLayer(H, L, scale=0.07), gen(6), sum(new)
    w, norm = (0.05 * randn(g, H, NOPE + V, L)).to(BF16), binding.make_latent_norm(THETA, EPS)
    per = [-(-x // PAGE) for x in new]

    class State:
        def __init__(self):
            self.table = torch.full((n, max(per)), -1, dtype=torch.int32, device="cuda")
            at = 0
            for b, k in enumerate(per):
                self.table[b, :k] = torch.arange(at, at + k, device="cuda")
                at += k
            self.pages = binding.make_pages(self.table, at)
            self.pool = torch.zeros(at, PAGE, L + R, dtype=torch.uint8 if fp8 else BF16, device="cuda")
            self.s8 = [torch.zeros(at, PAGE, device="cuda")] if fp8 else []
            self.ckv, self.q = randn(g, T, L + R).to(BF16), randn(g, T, H, NOPE + R).to(BF16)
            self.qa = randn(g, n, H, L + R).to(BF16)
            self.rot = self.q.clone()
            self.kv, self.rope = torch.empty(T, H, 256, dtype=BF16, device="cuda"), torch.empty(T, R, dtype=BF16, device="cuda")
            self.out, self.lse = torch.empty(T, H, V, dtype=BF16, device="cuda"), torch.empty(T, H, device="cuda")
            self.dec, self.ws = torch.empty(n, H, L, dtype=BF16, device="cuda"), binding.alloc_latent_workspace(layer, n)
            self.cu, self.past, self.len = cu(new), i32([0] * n), i32(new)

        def run(self, stream=None):
            write, expand, decode = ((binding.latent_norm_rope_cache_write_fp8, binding.latent_kv_expand_fp8, binding.attn_decode_latent_fp8) if fp8
                                     else (binding.latent_norm_rope_cache_write, binding.latent_kv_expand, binding.attn_decode_latent))
            write(layer, norm, self.ckv, self.q[..., NOPE:], self.cu, self.past, self.pages, self.rot[..., NOPE:], self.pool, *self.s8, stream=stream)
            expand(layer, self.pool, *self.s8, self.pages, self.cu, w, self.kv, self.rope, stream=stream)
            binding.attn_prefill_latent(layer, self.rot, self.cu, self.past, max(new), self.kv, self.rope, self.cu, self.out, self.lse, stream=stream)
            decode(layer, self.qa, self.pool, *self.s8, self.pages, self.len, self.dec, ws=self.ws, stream=stream)

        def outputs(self):
            return (self.pool, *self.s8, self.rot[..., NOPE:], self.kv, self.rope, self.out, self.lse, self.dec)

        def results(self):
            return [x.clone() for x in self.outputs()]

        def wipe(self):
            for x in self.outputs():
                x.zero_()

    a, b = State(), State()
    plain = []
    for s in (a, b):
        s.run()
        no_error()
        plain.append(s.results())
        pos = torch.cat([torch.arange(k, device="cuda") for k in new])
        want = rotated(s.q[..., NOPE:], pos)
        check(s.rot[..., NOPE:], want, H_BF16 * want.abs() + 2.0 ** -20 * rot_mag(s.q[..., NOPE:]), "queries")
        s.wipe()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for s, st in zip((a, b), streams):
            s.run(st)
    no_error()
    for s, want in zip((a, b), plain):
        assert all(torch.equal(x, y) for x, y in zip(s.results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    a.wipe()
    for x, y in ((a.ckv, b.ckv), (a.q, b.q), (a.qa, b.qa), (a.rot[..., :NOPE], b.rot[..., :NOPE])):
        x.copy_(y)
    for _ in range(3):
        graph.replay()
    no_error()
    assert all(torch.equal(x, y) for x, y in zip(a.results(), plain[1]))
