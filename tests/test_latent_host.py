"""Host-side checks of the latent-attention entry points that need no GPU:
workspace arithmetic and every refusal, before anything touches a device."""
import ctypes

import pytest

from paged_sliding_window_gb300 import binding, build
from paged_sliding_window_gb300.workloads import LatentLayer

FAKE = 0x10000  # aligned fake device address; validation never dereferences


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _layer(**kw):
    base = dict(n_heads=16, latent_dim=512, rope_dim=64, nope_dim=128, v_dim=128, window=0,
                softcap=0.0, scale=1.0, block_size=16)
    base.update(kw)
    return binding.PswLatent(**base)


def _pages(table=FAKE, mbps=64, nb=1024):
    return ctypes.byref(binding.PswPages(table, mbps, nb))


def _norm(theta=1e4, eps=1e-6, weight=None):
    return ctypes.byref(binding.PswLatentNorm(theta, eps, weight))


def call(lib, name, layer=None, **kw):
    """Every entry point with valid arguments except those given. n_seqs is 0 unless given, so
    that a call whose arguments pass returns before it asks for a device."""
    lp = ctypes.byref(layer or _layer())
    g = lambda k, d=FAKE: kw.get(k, d)  # noqa: E731
    pages = g("pages", _pages())
    n = g("n_seqs", 0)
    scale = [g("row_scale")] if name.endswith("fp8") else []
    if name.startswith("latent_norm"):
        return getattr(lib, name)(lp, g("norm", _norm()), g("ckv"), g("ckv_stride", 576), g("q"),
                                  g("qt", 16 * 192), g("qh", 192), g("cu"), g("past"), n, g("nt", 5), pages,
                                  g("qo", FAKE * 2), g("qot", 16 * 64), g("qoh", 64), g("pool"),
                                  *scale, None)
    if name.startswith("attn_decode"):
        return getattr(lib, name)(lp, g("q"), g("pool"), *scale, pages, g("seq"), n, g("out"),
                                  g("lse", None), g("ws"), g("ws_bytes", 1 << 40), None)
    if name.startswith("latent_kv"):
        return getattr(lib, name)(lp, g("pool"), *scale, pages, g("cu"), g("first", None), n,
                                  g("nk", 100), g("w"), g("kv"), g("rope"), None)
    return lib.attn_prefill_latent(lp, g("q"), g("cu"), g("past"), n, g("nq", 10), g("maxq", 10),
                                   g("kv"), g("rope"), g("cuk"), g("first", None), g("nk", 100),
                                   g("out"), g("lse", None), None)


WRITES = ["latent_norm_rope_cache_write", "latent_norm_rope_cache_write_fp8"]
DECODES = ["attn_decode_latent", "attn_decode_latent_fp8"]
EXPANDS = ["latent_kv_expand", "latent_kv_expand_fp8"]
PAGED = WRITES + DECODES + EXPANDS
EVERY = PAGED + ["attn_prefill_latent"]


@pytest.mark.parametrize("name", EVERY)
def test_valid_arguments_pass(lib, name):
    assert call(lib, name) == 0


@pytest.mark.parametrize("name", EVERY)
@pytest.mark.parametrize("kw,code", [
    (dict(n_heads=0), "PSW_EINVAL_HEADS"), (dict(n_heads=129), "PSW_EINVAL_HEADS"),
    (dict(n_heads=-1), "PSW_EINVAL_HEADS"), (dict(latent_dim=128), "PSW_EINVAL_HDIM"),
    (dict(latent_dim=513), "PSW_EINVAL_HDIM"), (dict(rope_dim=32), "PSW_EINVAL_HDIM"),
    (dict(nope_dim=64), "PSW_EINVAL_HDIM"), (dict(v_dim=256), "PSW_EINVAL_HDIM"),
    (dict(softcap=-1.0), "PSW_EINVAL_SOFTCAP"), (dict(softcap=float("nan")), "PSW_EINVAL_SOFTCAP"),
    (dict(window=-1), "PSW_EINVAL_WINDOW"), (dict(block_size=32), "PSW_EINVAL_BLOCKSIZE"),
    (dict(scale=0.0), "PSW_EINVAL_SCALE"), (dict(scale=float("inf")), "PSW_EINVAL_SCALE"),
])
def test_layer_refusals(lib, name, kw, code):
    got = call(lib, name, layer=_layer(**kw))
    assert binding.ERRORS.get(got) == code


@pytest.mark.parametrize("names,kw,code", [
    (WRITES, dict(norm=None), "PSW_ENULL"), (WRITES, dict(ckv=None), "PSW_ENULL"),
    (WRITES, dict(cu=None), "PSW_ENULL"), (WRITES, dict(past=None), "PSW_ENULL"),
    (WRITES, dict(pool=None), "PSW_ENULL"), (WRITES, dict(q=None), "PSW_ENULL"),
    (WRITES, dict(qo=None), "PSW_ENULL"), (WRITES, dict(norm=_norm(theta=0.0)), "PSW_EINVAL_ROPE"),
    (WRITES, dict(norm=_norm(eps=-1.0)), "PSW_EINVAL_ROPE"),
    (WRITES, dict(norm=_norm(theta=float("nan"))), "PSW_EINVAL_ROPE"),
    (WRITES, dict(ckv_stride=568), "PSW_EINVAL_STRIDE"), (WRITES, dict(ckv_stride=577), "PSW_EINVAL_STRIDE"),
    (WRITES, dict(nt=-1), "PSW_ECAPACITY"), (WRITES, dict(qh=60), "PSW_EINVAL_STRIDE"), (WRITES, dict(qot=68), "PSW_EINVAL_STRIDE"),
    (WRITES, dict(qoh=0), "PSW_EINVAL_STRIDE"), (WRITES, dict(qo=FAKE), "PSW_EINVAL_STRIDE"),
    (WRITES, dict(ckv=FAKE + 8), "PSW_EALIGN"), (WRITES, dict(q=FAKE + 2), "PSW_EALIGN"),
    (WRITES, dict(norm=_norm(weight=FAKE + 4)), "PSW_EALIGN"),
    (DECODES, dict(q=None), "PSW_ENULL"), (DECODES, dict(seq=None), "PSW_ENULL"),
    (DECODES, dict(out=None), "PSW_ENULL"), (DECODES, dict(out=FAKE + 8), "PSW_EALIGN"),
    (DECODES, dict(ws=FAKE + 8), "PSW_EALIGN"), (DECODES, dict(lse=FAKE + 2), "PSW_EALIGN"),
    (DECODES, dict(n_seqs=1 << 20, pages=_pages(mbps=1 << 12)), "PSW_ECAPACITY"),
    (DECODES, dict(n_seqs=4, ws=None), "PSW_EWORKSPACE"),
    (DECODES, dict(n_seqs=4, ws_bytes=100), "PSW_EWORKSPACE"),
    (EXPANDS, dict(w=None), "PSW_ENULL"), (EXPANDS, dict(kv=None), "PSW_ENULL"),
    (EXPANDS, dict(rope=None), "PSW_ENULL"), (EXPANDS, dict(cu=None), "PSW_ENULL"),
    (EXPANDS, dict(nk=-1), "PSW_ECAPACITY"), (EXPANDS, dict(w=FAKE + 8), "PSW_EALIGN"),
    (PAGED, dict(pool=None), "PSW_ENULL"), (PAGED, dict(pages=None), "PSW_ENULL"),
    (PAGED, dict(pages=_pages(table=None)), "PSW_ENULL"), (PAGED, dict(pages=_pages(mbps=0)), "PSW_ECAPACITY"),
    (PAGED, dict(pages=_pages(nb=(1 << 27) + 1)), "PSW_ECAPACITY"),
    (PAGED, dict(n_seqs=-1), "PSW_EINVAL_NSEQS"), (PAGED, dict(pool=FAKE + 8), "PSW_EALIGN"),
    (["attn_prefill_latent"], dict(q=None), "PSW_ENULL"), (["attn_prefill_latent"], dict(kv=None), "PSW_ENULL"),
    (["attn_prefill_latent"], dict(cuk=None), "PSW_ENULL"), (["attn_prefill_latent"], dict(out=None), "PSW_ENULL"),
    (["attn_prefill_latent"], dict(kv=None, rope=None, nk=0), "PSW_OK"),
    (["attn_prefill_latent"], dict(n_seqs=65536), "PSW_EINVAL_NSEQS"),
    (["attn_prefill_latent"], dict(n_seqs=-1), "PSW_EINVAL_NSEQS"),
    (["attn_prefill_latent"], dict(maxq=-1), "PSW_ECAPACITY"),
    (["attn_prefill_latent"], dict(kv=FAKE + 8), "PSW_EALIGN"),
])
def test_argument_refusals(lib, names, kw, code):
    for name in names:
        got = call(lib, name, **kw)
        assert {0: "PSW_OK", **binding.ERRORS}.get(got) == code, name


def test_fp8_calls_need_their_scales(lib):
    for name in ("latent_norm_rope_cache_write_fp8", "attn_decode_latent_fp8", "latent_kv_expand_fp8"):
        assert binding.ERRORS[call(lib, name, row_scale=None)] == "PSW_ENULL"
        assert binding.ERRORS[call(lib, name, row_scale=FAKE + 2)] == "PSW_EALIGN"


def test_workspace_bytes(lib):
    assert binding.latent_workspace_bytes(LatentLayer(16), 0) >= 0
    assert binding.latent_workspace_bytes(LatentLayer(128), 64) >= binding.latent_workspace_bytes(LatentLayer(16), 64)
    with pytest.raises(binding.PswError) as e:
        binding.latent_workspace_bytes(LatentLayer(16), -1)
    assert binding.ERRORS[e.value.code] == "PSW_EINVAL_NSEQS"


def test_layer_structs_are_shared_by_value():
    assert binding.make_latent_layer(LatentLayer(16)) is binding.make_latent_layer(LatentLayer(16))
    assert binding.make_latent_layer(LatentLayer(16)) is not binding.make_latent_layer(LatentLayer(17))
