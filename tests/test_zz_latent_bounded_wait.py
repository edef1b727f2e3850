"""The latent decode's bounded waits, made to run out in the allowed way: the
testing hook has one CTA leave a tile unasked for, so that the waits for it end
at their bound. What that CTA should have noted for the join is then missing,
and the workspace, which needs no zeroing, holds anything in its place: the join
must not form addresses from it. The call comes back with PSW_DEVERR_PIPELINE,
and the next one on the same buffers gives the bits of the one before."""
import time

import pytest
import torch

from latent_harness import BF16, LatentLayer, i32, no_error
from paged_sliding_window_gb300 import binding
from test_gpu_latent import _decode_call, _decode_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def hook_off():
    binding.testing_stall(binding.STALL_OFF)
    yield
    binding.testing_stall(binding.STALL_OFF)


# pieces (first, last) that the workspace claims for every unit
@pytest.mark.parametrize("claim", [(0x7F7F7F7F, 0x7F7F7F7F), (3, 0x40000000), (0, 1 << 20), (150, 4)],
                         ids=["far", "long", "many", "reversed"])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_wait_runs_out(fp8, claim):
    layer, lens = LatentLayer(16, 512, scale=0.07), [60000, 100, 0]  # several tiles for every CTA
    pg, q = _decode_inputs(layer, lens, fp8, 3)
    lens_t, ws = i32(lens), binding.alloc_latent_workspace(layer, len(lens))

    def call():
        out, lse = torch.zeros(3, 16, 512, dtype=BF16, device="cuda"), torch.zeros(3, 16, device="cuda")
        _decode_call(layer, pg, q, lens_t, out, lse, ws)
        return out, lse

    plain = call()
    no_error()
    ws[:len(lens) * 8].view(torch.int32).view(-1, 2).copy_(i32([claim] * len(lens)))
    torch.cuda.synchronize()
    binding.testing_stall(binding.STALL_DECODE, 0, 2)
    t0 = time.time()
    call()
    err = binding.get_error()
    elapsed = time.time() - t0
    binding.testing_stall(binding.STALL_OFF)
    assert err & binding.DEVERR_PIPELINE, err
    assert 0.3 < elapsed < 30, elapsed
    again = call()  # allocates tensor memory on every SM again
    no_error()
    for a, b in zip(plain, again):
        assert torch.equal(a, b)
