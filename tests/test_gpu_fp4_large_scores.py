"""The 4-bit decode with scores so large that fp32 has steps of several units there: weights stay within
what fp16 holds."""
import pytest
import torch

from fp4_harness import BF16, Cache, Layer, S_ERR, check, gen, no_error, normed
from paged_sliding_window_gb300 import binding
from test_gpu_fp4 import decode

pytestmark = pytest.mark.gpu


SEQS, KEYS, EACH, DIGITS = 600, 2000, 32, 6


@pytest.mark.parametrize("power", [10, 12, 13, 14, 15, 16, 17, 20])
@pytest.mark.parametrize("unit", [0.5, 1.0, 1.5, 2.0])
@pytest.mark.parametrize("layer", [Layer(2, 1, 256), Layer(4, 1, 256, k_eq_v=True), Layer(2, 1, 512), Layer(4, 1, 512, k_eq_v=True)],
                         ids=["256", "256-keqv", "512", "512-keqv"])
def test_scores_that_grow_by_single_steps(layer, unit, power):
    """Scores 2688 2^power + 6 unit (j / 32) of keys j, from a few powers of two below where fp32's steps pass
    1 to a few above. All keys have the same values (where they are keys too, all but the digits of
    j / 32), so the result is those, whatever the weights; and the sum of the weights is that of 64 bits
    within the steps of the scores. Sequences share one context, so that many pages are worked on in a row."""
    hd = layer.head_dim
    j = torch.arange(KEYS, device="cuda") // EACH
    k = torch.zeros(KEYS, 1, hd, device="cuda")
    k[:, 0, 0] = 2688  # the largest value there is
    for i in range(DIGITS):  # (alone in their blocks: exact)
        k[:, 0, 16 * (1 + i)] = 6.0 * (j >> i & 1)
    rest = slice(16 * (1 + DIGITS), hd)
    k[..., rest] = normed(gen(80), 1, hd - rest.start).float()
    cache = Cache(layer, [KEYS], 80)
    v = None if layer.k_eq_v else normed(gen(81), 1, 1, hd).expand(KEYS, -1, -1).contiguous()
    cache.write(k.to(BF16), v, [KEYS], [0])
    cache.table = cache.table.expand(SEQS, -1).contiguous()
    cache.pages = binding.make_pages(cache.table, cache.blocks)
    size = torch.tensor([1.0, 0.5, 0.25, 1.0], device="cuda")[:layer.n_q_heads]
    q = torch.zeros(SEQS, layer.n_q_heads, hd, device="cuda")
    q[..., 0] = 2.0 ** power * size
    for i in range(DIGITS):
        q[..., 16 * (1 + i)] = unit * 2.0 ** i * size
    lens = [KEYS - (b % 5) * 37 for b in range(SEQS)]
    out, lse = decode(layer, cache, q.to(BF16), lens)
    no_error()
    assert bool(out.isfinite().all())
    want = cache.rows(cache.k if v is None else cache.v, 0, 0, 1, 1.0)[0, 0]
    keep = torch.ones(hd, dtype=torch.bool, device="cuda")
    if v is None:
        keep[16:rest.start] = False
    # the weights are rounded one by one, their sum is not: 2^-11 at most, and the result to bf16
    check(out[..., keep], want[keep].expand(*out.shape[:2], -1), want[keep].abs() * (2.0 ** -8 + 2.0 ** -10), "out")
    s = (2688.0 * 2.0 ** power + 6 * unit * j.double()) * size[:, None].double()
    for n in set(lens):
        rows = [b for b in range(SEQS) if lens[b] == n]
        ref = torch.logsumexp(s[:, :n], -1)
        check(lse[rows], ref.expand(len(rows), -1), (ref.abs() * S_ERR).expand(len(rows), -1), "lse")
