"""The latent-attention operators where offsets pass 32 bits, and all of them in one captured
graph. What lies far is compared bit for bit with the same work on small tensors, which the
other parity tests compare with 64 bits."""
import pytest
import torch

from latent_harness import BF16, EPS, NOPE, R, THETA, V, LatentLayer, binding, cu, gen, i32, no_error, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_far_pages(fp8):
    """Pages whose first value has an index beyond 2^31."""
    L, H, lens = 512, 8, [70, 200]
    layer, g, T = LatentLayer(H, L, scale=0.05), gen(3), sum(lens)
    far = 2 ** 31 // (16 * (L + R)) + 1
    total = far + 20
    dtype = torch.uint8 if fp8 else BF16
    ckv, w = randn(g, T, L + R).to(BF16), (0.05 * randn(g, H, NOPE + V, L)).to(BF16)
    q, qs = randn(g, 2, H, L + R).to(BF16), randn(g, T, H, R).to(BF16)
    ids = torch.randperm(20, generator=g, device="cuda").to(torch.int32)[:18]
    got = []
    for first, blocks in ((0, 20), (far, total)):
        pool = torch.empty(blocks, 16, L + R, dtype=dtype, device="cuda")
        scale = torch.empty(blocks, 16, device="cuda") if fp8 else None
        table = torch.full((2, 13), -1, dtype=torch.int32, device="cuda")
        table[0, :5], table[1, :13] = ids[:5] + first, ids[5:18] + first
        pages, qo, s8 = binding.make_pages(table, blocks), torch.empty_like(qs), [scale] if fp8 else []
        write, decode, expand = ((binding.latent_norm_rope_cache_write_fp8, binding.attn_decode_latent_fp8, binding.latent_kv_expand_fp8)
                                 if fp8 else (binding.latent_norm_rope_cache_write, binding.attn_decode_latent, binding.latent_kv_expand))
        write(layer, binding.make_latent_norm(THETA, EPS), ckv, qs, cu(lens), i32([0, 0]), pages, qo, pool, *s8)
        out, lse = torch.empty(2, H, L, dtype=BF16, device="cuda"), torch.empty(2, H, device="cuda")
        decode(layer, q, pool, *s8, pages, i32(lens), out, lse, ws=binding.alloc_latent_workspace(layer, 2))
        kv, rope = torch.empty(T, H, 256, dtype=BF16, device="cuda"), torch.empty(T, R, dtype=BF16, device="cuda")
        expand(layer, pool, *s8, pages, cu(lens), w, kv, rope)
        no_error()
        got.append((out, lse, kv, rope, qo))
        del pool
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_far_rows():
    """Queries, keys, values and results beyond 2^31 values: 300 rows behind 131072 without keys,
    their keys behind 66000 of a sequence without rows."""
    H, rows, keys = 128, 300, 500
    layer, g = LatentLayer(H, scale=0.05), gen(4)
    q0, k0 = 131072, 66000
    q, kv, rope = randn(g, rows, H, NOPE + R).to(BF16), randn(g, keys, H, NOPE + V).to(BF16), randn(g, keys, R).to(BF16)
    out, lse = torch.empty(rows, H, V, dtype=BF16, device="cuda"), torch.empty(rows, H, device="cuda")
    binding.attn_prefill_latent(layer, q, cu([rows]), i32([keys - rows]), rows, kv, rope, cu([keys]), out, lse)
    qf = torch.zeros(q0 + rows, H, NOPE + R, dtype=BF16, device="cuda")
    kvf = torch.zeros(k0 + keys, H, NOPE + V, dtype=BF16, device="cuda")
    rf = torch.zeros(k0 + keys, R, dtype=BF16, device="cuda")
    qf[q0:], kvf[k0:], rf[k0:] = q, kv, rope
    outf = torch.full((q0 + rows, H, V), 3.0, dtype=BF16, device="cuda")
    lsef = torch.empty(q0 + rows, H, device="cuda")
    binding.attn_prefill_latent(layer, qf, cu([q0, 0, rows]), i32([0, 0, keys - rows]), q0, kvf, rf, cu([0, k0, keys]), outf, lsef)
    no_error()
    assert torch.equal(outf[q0:], out) and torch.equal(lsef[q0:], lse)
    assert bool((outf[:q0] == 0).all()) and bool(torch.isneginf(lsef[:q0]).all())


def test_far_expansion():
    """Expanded rows beyond 2^31 values: the last rows of 70000 equal those expanded alone."""
    L, H, n, last = 256, 128, 70000, 100
    layer, g = LatentLayer(H, L), gen(5)
    blocks = -(-n // 16)
    pool, w = randn(g, blocks, 16, L + R).to(BF16), (0.06 * randn(g, H, NOPE + V, L)).to(BF16)
    pages = binding.make_pages(torch.arange(blocks, dtype=torch.int32, device="cuda")[None].contiguous(), blocks)
    kv, rope = torch.empty(n, H, 256, dtype=BF16, device="cuda"), torch.empty(n, R, dtype=BF16, device="cuda")
    binding.latent_kv_expand(layer, pool, pages, cu([n]), w, kv, rope)
    a, b = torch.empty(last, H, 256, dtype=BF16, device="cuda"), torch.empty(last, R, dtype=BF16, device="cuda")
    binding.latent_kv_expand(layer, pool, pages, cu([last]), w, a, b, k_first=i32([n - last]))
    no_error()
    assert torch.equal(kv[-last:], a) and torch.equal(rope[-last:], b)


@pytest.mark.parametrize("H,new", [(4, [150, 33]), (48, [90, 200]), (4, [600, 20]), (48, [600, 300, 513]), (64, [90] * 12)],
                         ids=["spare-pairs", "singles", "pairs", "many-pairs", "many-singles"])
def test_chain_captured(H, new):
    """Write, expansion, chunk attention and decode in one graph, replayed with other inputs, and
    on two streams at once; each gives what the calls give one by one."""
    L, n = 512, len(new)
    layer, g, T = LatentLayer(H, L, scale=0.07), gen(6), sum(new)
    w, norm = (0.05 * randn(g, H, NOPE + V, L)).to(BF16), binding.make_latent_norm(THETA, EPS)
    per = [-(-x // 16) for x in new]

    class State:
        def __init__(self):
            self.table = torch.full((n, max(per)), -1, dtype=torch.int32, device="cuda")
            at = 0
            for b, k in enumerate(per):
                self.table[b, :k] = torch.arange(at, at + k, device="cuda")
                at += k
            self.pages = binding.make_pages(self.table, at)
            self.pool = torch.zeros(at, 16, L + R, dtype=BF16, device="cuda")
            self.ckv, self.q = randn(g, T, L + R).to(BF16), randn(g, T, H, NOPE + R).to(BF16)
            self.qa = randn(g, n, H, L + R).to(BF16)
            self.rot = torch.empty_like(self.q)
            self.kv, self.rope = torch.empty(T, H, 256, dtype=BF16, device="cuda"), torch.empty(T, R, dtype=BF16, device="cuda")
            self.out, self.lse = torch.empty(T, H, V, dtype=BF16, device="cuda"), torch.empty(T, H, device="cuda")
            self.dec, self.ws = torch.empty(n, H, L, dtype=BF16, device="cuda"), binding.alloc_latent_workspace(layer, n)
            self.cu, self.past, self.len = cu(new), i32([0] * n), i32(new)

        def run(self, stream=None):
            binding.latent_norm_rope_cache_write(layer, norm, self.ckv, self.q[..., NOPE:], self.cu, self.past, self.pages,
                                                 self.rot[..., NOPE:], self.pool, stream=stream)
            binding.latent_kv_expand(layer, self.pool, self.pages, self.cu, w, self.kv, self.rope, stream=stream)
            binding.attn_prefill_latent(layer, self.q, self.cu, self.past, max(new), self.kv, self.rope, self.cu, self.out, self.lse, stream=stream)
            binding.attn_decode_latent(layer, self.qa, self.pool, self.pages, self.len, self.dec, ws=self.ws, stream=stream)

        def results(self):
            return [x.clone() for x in (self.pool, self.kv, self.rope, self.out, self.lse, self.dec)]

    a, b = State(), State()
    plain = []
    for s in (a, b):
        s.run()
        torch.cuda.synchronize()
        plain.append(s.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in (a, b):
        for x in (s.pool, s.kv, s.rope, s.out, s.lse, s.dec):
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for s, st in zip((a, b), streams):
            s.run(st)
    torch.cuda.synchronize()
    no_error()
    for s, want in zip((a, b), plain):
        assert all(torch.equal(x, y) for x, y in zip(s.results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for x, y in ((a.ckv, b.ckv), (a.q, b.q), (a.qa, b.qa)):
        x.copy_(y)
    for _ in range(3):
        graph.replay()
    no_error()
    assert all(torch.equal(x, y) for x, y in zip(a.results(), plain[1]))
