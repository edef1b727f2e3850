"""A sequence whose past length is negative gets no row of a 4-bit cache write, not those of its tokens
that would come to a position either."""
import pytest
import torch

from fp4_harness import Cache, Layer, cu, gen, i32, normed, quantised, takes_error
from paged_sliding_window_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("past", [-1, -7, -2 ** 31])
@pytest.mark.parametrize("others", [1, 40], ids=["few", "many"])  # (sequences are looked up otherwise beyond 31)
@pytest.mark.parametrize("layer", [Layer(4, 2, 256), Layer(6, 3, 512, k_eq_v=True)], ids=["256", "512-keqv"])
def test_write_leaves_out_a_sequence_with_a_negative_past(layer, others, past):
    new, pasts = [3] * others + [40], [5] * others + [past]
    cache, g = Cache(layer, [8] * others + [48], 50), gen(50)
    k = normed(g, sum(new), layer.n_kv_heads, layer.head_dim)
    v = None if layer.k_eq_v else normed(g, *k.shape)
    fresh = cache.k[cache.table[others, :3].long()].clone()
    binding.kv_cache_write_fp4(layer, k, v, cu(new), i32(pasts), cache.pages, cache.k, cache.v)
    takes_error(binding.DEVERR_LENGTH)
    for x, pool in ((k, cache.k), (v, cache.v)):
        if x is None:
            continue
        assert torch.equal(pool[cache.table[others, :3].long()], fresh)
        for b in range(others):
            assert torch.equal(cache.rows(pool, b, 5, 8, 1.0), quantised(x[3 * b:3 * b + 3], 1.0))
