"""Host-side checks of the 4-bit pages' and the device tables' entry points that need no GPU:
workspace arithmetic and every refusal, before anything touches a device."""
import ctypes
import os
import re

import pytest

from paged_sliding_window_gb300 import binding, build

FAKE = 0x10000  # aligned fake device address; validation never dereferences
HEADER = os.path.join(build.ROOT, "include", "psw.h")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _layer(**kw):
    base = dict(n_q_heads=16, n_kv_heads=8, head_dim=256, window=0, softcap=0.0, scale=1.0, k_eq_v=0, block_size=16)
    base.update(kw)
    return binding.PswLayer(**base)


def _pages(table=FAKE, mbps=64, nb=1024):
    return ctypes.byref(binding.PswPages(table, mbps, nb))


def call(lib, name, layer=None, **kw):
    """Every entry point with valid arguments except those given. n_seqs is 0 unless given, so that a call
    whose arguments pass returns before it asks for a device."""
    z = layer or _layer()
    g = lambda k, d=FAKE: kw.get(k, d)  # noqa: E731
    vp = None if z.k_eq_v else FAKE
    lp, n = g("layer_ptr", ctypes.byref(z)), g("n", 0)
    if name == "write":
        return lib.kv_cache_write_fp4(lp, g("k"), g("v", vp), g("cu"), g("past"), n, g("rows", 5), g("pages", _pages()),
                                      g("kp"), g("vp", vp), g("ks", 1.0), g("vs", 1.0), None)
    if name == "read":
        return lib.kv_cache_read_fp4(lp, g("kp"), g("vp", vp), g("pages", _pages()), g("first", None), g("seq"), n,
                                     g("out_pages", _pages()), g("k"), g("v", vp), g("ks", 1.0), g("vs", 1.0), None)
    return lib.attn_decode_paged_fp4(lp, g("q"), g("kp"), g("vp", vp), g("pages", _pages()), g("seq"), n, g("out"),
                                     g("lse", None), g("ws"), g("ws_bytes", 1 << 40), g("ks", 1.0), g("vs", 1.0), None)


def tables(lib, **kw):
    g = lambda k, d=FAKE: kw.get(k, d)  # noqa: E731
    return lib.block_table_extend(g("table"), g("mbps", 64), g("past"), g("new"), g("n", 0), g("free"), g("n_free", 10), g("pos"),
                                  g("next"), g("cu"), g("lens"), g("slots"), g("n_slots", 5), None)


EVERY = ["write", "read", "decode"]


@pytest.mark.parametrize("name", EVERY)
@pytest.mark.parametrize("keqv", [0, 1])
def test_valid_arguments_pass(lib, name, keqv):
    assert call(lib, name, _layer(k_eq_v=keqv)) == 0
    assert call(lib, name, _layer(k_eq_v=keqv, head_dim=512)) == 0
    assert tables(lib) == 0 and tables(lib, slots=None) == 0 and tables(lib, free=None, n_free=0) == 0


@pytest.mark.parametrize("name", EVERY)
@pytest.mark.parametrize("kw,code", [
    (dict(n_q_heads=0), "PSW_EINVAL_HEADS"), (dict(n_q_heads=15), "PSW_EINVAL_HEADS"), (dict(n_kv_heads=-1), "PSW_EINVAL_HEADS"),
    (dict(head_dim=128), "PSW_EINVAL_HDIM"), (dict(softcap=-1.0), "PSW_EINVAL_SOFTCAP"), (dict(softcap=float("nan")), "PSW_EINVAL_SOFTCAP"),
    (dict(window=-1), "PSW_EINVAL_WINDOW"), (dict(block_size=32), "PSW_EINVAL_BLOCKSIZE"), (dict(scale=0.0), "PSW_EINVAL_SCALE"),
    (dict(scale=float("inf")), "PSW_EINVAL_SCALE"), (dict(k_eq_v=3), "PSW_EINVAL_KEQV"),
])
def test_layer_refusals(lib, name, kw, code):
    assert binding.ERRORS[call(lib, name, _layer(**kw))] == code
    size = ctypes.c_size_t(0)
    assert binding.ERRORS[lib.psw_fp4_workspace_bytes(ctypes.byref(_layer(**kw)), 3, ctypes.byref(size))] == code


@pytest.mark.parametrize("name,kw,code", [
    *[(e, dict(layer_ptr=None), "PSW_ENULL") for e in EVERY], *[(e, dict(pages=None), "PSW_ENULL") for e in EVERY],
    *[(e, dict(pages=_pages(table=None)), "PSW_ENULL") for e in EVERY], *[(e, dict(pages=_pages(mbps=0)), "PSW_ECAPACITY") for e in EVERY],
    *[(e, dict(pages=_pages(nb=(1 << 27) + 1)), "PSW_ECAPACITY") for e in EVERY], *[(e, dict(n=-1), "PSW_EINVAL_NSEQS") for e in EVERY],
    *[(e, dict(kp=None), "PSW_ENULL") for e in EVERY], *[(e, dict(vp=None), "PSW_EINVAL_KEQV") for e in EVERY],
    *[(e, dict(kp=FAKE + 8), "PSW_EALIGN") for e in EVERY], *[(e, dict(vp=FAKE + 4), "PSW_EALIGN") for e in EVERY],
    *[(e, {x: s}, "PSW_EINVAL_SCALE") for e in EVERY for x in ("ks", "vs") for s in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 61, 2.0 ** -61)],
    *[("write", {x: None}, "PSW_ENULL") for x in ("k", "cu", "past")], ("write", dict(v=None), "PSW_EINVAL_KEQV"),
    ("write", dict(rows=-1), "PSW_ECAPACITY"), ("write", dict(k=FAKE + 2), "PSW_EALIGN"), ("write", dict(v=FAKE + 2), "PSW_EALIGN"),
    ("read", dict(seq=None), "PSW_ENULL"), ("read", dict(k=None), "PSW_ENULL"), ("read", dict(v=None), "PSW_EINVAL_KEQV"),
    ("read", dict(out_pages=None), "PSW_ENULL"), ("read", dict(out_pages=_pages(nb=0)), "PSW_ECAPACITY"), ("read", dict(k=FAKE + 8), "PSW_EALIGN"),
    ("read", dict(n=1 << 20, pages=_pages(mbps=1 << 11)), "PSW_ECAPACITY"),
    *[("decode", {x: None}, "PSW_ENULL") for x in ("q", "seq", "out")], ("decode", dict(q=FAKE + 8), "PSW_EALIGN"),
    ("decode", dict(out=FAKE + 8), "PSW_EALIGN"), ("decode", dict(lse=FAKE + 2), "PSW_EALIGN"), ("decode", dict(ws=FAKE + 8), "PSW_EALIGN"),
    ("decode", dict(n=1, ws=None), "PSW_EWORKSPACE"), ("decode", dict(n=1, ws_bytes=100), "PSW_EWORKSPACE"),
    ("decode", dict(n=1 << 20, pages=_pages(mbps=1 << 8)), "PSW_ECAPACITY"),
])
def test_argument_refusals(lib, name, kw, code):
    assert binding.ERRORS[call(lib, name, **kw)] == code


def test_k_eq_v_takes_no_values(lib):
    for name, kw in (("write", dict(v=FAKE)), ("write", dict(vp=FAKE)), ("read", dict(v=FAKE)), ("read", dict(vp=FAKE)), ("decode", dict(vp=FAKE))):
        assert binding.ERRORS[call(lib, name, _layer(k_eq_v=1), **kw)] == "PSW_EINVAL_KEQV"


@pytest.mark.parametrize("kw,code", [
    *[({x: None}, "PSW_ENULL") for x in ("table", "past", "new", "free", "pos", "next", "cu", "lens")],
    *[({x: FAKE + 2}, "PSW_EALIGN") for x in ("table", "past", "new", "free", "pos", "next", "cu", "lens")], (dict(slots=FAKE + 4), "PSW_EALIGN"),
    (dict(n=-1), "PSW_EINVAL_NSEQS"), (dict(mbps=0), "PSW_ECAPACITY"), (dict(n_free=-1), "PSW_ECAPACITY"), (dict(n_slots=-1), "PSW_ECAPACITY"),
    (dict(mbps=1 << 27), "PSW_ECAPACITY"), (dict(n=1 << 20, mbps=1 << 11), "PSW_ECAPACITY"),
])
def test_table_refusals(lib, kw, code):
    assert binding.ERRORS[tables(lib, **kw)] == code


def test_workspace_and_constants(lib):
    """Counters, then slots of partial rows and their (m, l): one per warp and CTA of the largest grid and per unit."""
    text = open(HEADER).read()
    assert int(re.search(r"#define\s+PSW_FP4_COUNTER_BYTES\s+(\d+)", text).group(1)) == binding.FP4_COUNTER_BYTES
    assert int(re.search(r"#define\s+PSW_DEVERR_NOBLOCKS\s+(\d+)", text).group(1)) == binding.DEVERR_NOBLOCKS
    for layer, n in ((_layer(), 64), (_layer(n_q_heads=32, n_kv_heads=4, head_dim=512), 7), (_layer(n_q_heads=22, n_kv_heads=2), 0)):
        G = layer.n_q_heads // layer.n_kv_heads
        units = n * layer.n_kv_heads * -(-G // 8)
        rows = (min(G, 8) + 1) // 2 * 2
        assert binding.fp4_workspace_bytes(layer, n) == 16384 + (160 * 13 + units) * rows * (4 * layer.head_dim + 8 * 8)
    assert binding.fp4_page_bytes(_layer()) == 2304


@pytest.mark.skipif(os.path.exists("/dev/nvidia0"), reason="host without a GPU only")
def test_valid_call_without_gpu_fails_loudly(lib):
    for name in EVERY:
        assert binding.ERRORS[call(lib, name, n=2)] == "PSW_EDEVICE"
    assert binding.ERRORS[tables(lib, n=2)] == "PSW_EDEVICE"
