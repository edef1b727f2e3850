"""The 4-bit decode with a softcap far below the scores, large tensor scales and rows of zeros: a score of 0
stays 0 where the scores' factor is beyond fp32."""
import pytest
import torch

from fp4_harness import BF16, Cache, Layer, gen, no_error, normed
from test_gpu_fp4 import compare, decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap,gs", [(1e-30, 2.0 ** 60), (1e-12, 2.0 ** 60), (1e-30, 1.0), (1e-6, 2.0 ** 40)])
@pytest.mark.parametrize("hd,k_eq_v", [(256, False), (256, True), (512, False), (512, True)])
def test_zero_rows_under_a_small_cap(hd, k_eq_v, softcap, gs):
    layer, lens, g = Layer(8, 2, hd, scale=1.0, softcap=softcap, k_eq_v=k_eq_v), [130, 40], gen(70)
    cache, n = Cache(layer, lens, 70), sum(lens)
    k = (normed(g, n, 2, hd).float() * gs).to(BF16)
    k[::3] = 0
    v = None if k_eq_v else normed(g, n, 2, hd)
    cache.write(k, v, lens, [0, 0], (gs, 1.0))
    q = normed(g, 2, 8, hd)
    q[1, 3] = 0
    got = decode(layer, cache, q, lens, (gs, 1.0))
    no_error()
    assert bool(got[0].isfinite().all()) and bool(got[1].isfinite().all())
    compare(layer, cache, q, lens, got, (gs, 1.0))
