"""The struct that make_latent_layer hands out is shared: nobody can change it under the others."""
import copy

import pytest

from paged_sliding_window_gb300 import binding
from paged_sliding_window_gb300.workloads import LatentLayer


def fields(z):
    return {name: getattr(z, name) for name, _ in binding.PswLatent._fields_}


def test_a_returned_struct_cannot_change_later_calls():
    layer = LatentLayer(16, 512, window=128, softcap=30.0, scale=0.25)
    z = binding.make_latent_layer(layer)
    want = dict(n_heads=16, latent_dim=512, rope_dim=64, nope_dim=128, v_dim=128, window=128, softcap=30.0, scale=0.25, block_size=16)
    assert fields(z) == want
    for name in want:
        with pytest.raises(AttributeError):
            setattr(z, name, 64)
    assert fields(binding.make_latent_layer(layer)) == want


def test_own_structs_stay_the_callers():
    z = binding.PswLatent(4, 256, 64, 128, 128, 0, 0.0, 1.0, 16)
    assert binding.make_latent_layer(z) is z
    z.window = 7
    assert binding.make_latent_layer(z).window == 7
    # a copy of a shared one by its fields is one's own as well
    own = binding.PswLatent(*fields(binding.make_latent_layer(LatentLayer(16))).values())
    own.window = 7
    assert binding.make_latent_layer(LatentLayer(16)).window == 0
    assert binding.latent_workspace_bytes(own, 2) == binding.latent_workspace_bytes(LatentLayer(16), 2)
    assert fields(copy.copy(own)) == fields(own)
