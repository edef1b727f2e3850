"""A bounded wait of the 4-bit decode made to run out (testing hook psw_testing_stall): one warp's page
is not asked for, nothing faults or spins without a bound, the call returns with an error bit, and the next
call, its workspace's counters zeroed, is exact."""
import time

import pytest
import torch

from fp4_harness import BF16, Layer, no_error
from paged_sliding_window_gb300 import binding
from test_gpu_fp4 import compare, decode, filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cta,tile", [(0, 0), (1, 2), (3, 1)])
@pytest.mark.parametrize("layer", [Layer(4, 2, 256), Layer(8, 1, 512, k_eq_v=True)], ids=["256", "512-keqv"])
def test_wait_runs_out_and_the_next_call_is_exact(layer, cta, tile):
    run_out(layer, [38000, 30000, 40, 120000], cta, tile)  # (several tiles for every warp)


@pytest.mark.parametrize("cta", [0, 2])
@pytest.mark.parametrize("layer", [Layer(4, 2, 256), Layer(4, 2, 512, k_eq_v=True)], ids=["256", "512-keqv"])
def test_wait_runs_out_where_a_block_has_a_unit(layer, cta):
    run_out(layer, [300, 40], cta, 0)


def run_out(layer, lens, cta, tile):
    cache, q = filled(layer, lens, 41)
    ws = binding.alloc_fp4_workspace(layer, len(lens))
    want = decode(layer, cache, q, lens, ws=ws)
    no_error()
    compare(layer, cache, q, lens, want)
    binding.testing_stall(binding.STALL_DECODE, cta, tile)
    try:
        begin = time.monotonic()
        decode(layer, cache, q, lens, ws=ws)
        torch.cuda.synchronize()
        took = time.monotonic() - begin
    finally:
        binding.testing_stall(binding.STALL_OFF)
    assert binding.get_error() == binding.DEVERR_PIPELINE
    assert 0.3 < took < 30
    ws[:binding.FP4_COUNTER_BYTES].zero_()
    got = decode(layer, cache, q, lens, ws=ws)
    no_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].dtype == BF16
    assert bool((ws[:binding.FP4_COUNTER_BYTES] == 0).all())
