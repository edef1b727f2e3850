"""The checks of tensors in the binding of the 4-bit pages and the device tables, one wrong tensor at a time,
without a GPU: the tensors are stand-ins that say where they are, the library one that counts its calls."""
import pytest
import torch

from paged_sliding_window_gb300 import binding
from paged_sliding_window_gb300.workloads import Layer

I32, F32, BF16, U8, I64 = torch.int32, torch.float32, torch.bfloat16, torch.uint8, torch.int64


class Tensor:
    """A tensor on a device: what the binding asks one, and nothing behind it."""

    def __init__(self, dtype, *shape, device=0, packed=True):
        self.dtype, self.shape, self.place, self.packed = dtype, torch.Size(shape), device, packed
        self.is_cuda = device >= 0
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")

    def numel(self):
        return self.shape.numel()

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.place

    def is_contiguous(self):
        return self.packed

    def data_ptr(self):
        return 0x10000 if self.numel() else 0


class Library:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*a):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(binding, "load", lambda *a: lib)
    monkeypatch.setattr(binding, "_stream_here", lambda device, stream: 0)
    return lib


def pages(table, blocks):
    p = binding.PswPages(table.data_ptr(), table.shape[1], blocks)
    p.table = table
    return p


N, ROWS, KV, HD, BLOCKS = 3, 7, 2, 256, 11


def cases(name, k_eq_v):
    """(call, {argument: (dtype, shape)}) with every tensor of the call."""
    layer = Layer(4, KV, HD, k_eq_v=k_eq_v)
    rows, pool, wide = (BF16, (ROWS, KV, HD)), (U8, (BLOCKS, KV, 9 * HD)), (BF16, (BLOCKS, 16, KV, HD))
    each, table = (I32, (N,)), (I32, (N, 5))
    v = lambda x: {} if k_eq_v else x  # noqa: E731
    if name == "tables":
        return (lambda t: binding.block_table_extend(*(t[x] for x in ("table", "past", "new", "free", "pos", "next", "cu", "lens", "slots"))),
                dict(table=table, past=each, new=each, free=(I32, (9,)), pos=(I32, (1,)), next=(I32, (1,)), cu=(I32, (N + 1,)), lens=each, slots=(I64, (8,))))
    if name == "write":
        return (lambda t: binding.kv_cache_write_fp4(layer, t["k"], t.get("v"), t["cu"], t["past"], pages(t["table"], BLOCKS), t["kp"], t.get("vp")),
                dict(k=rows, cu=(I32, (N + 1,)), past=each, table=table, kp=pool, **v(dict(v=rows, vp=pool))))
    if name == "read":
        return (lambda t: binding.kv_cache_read_fp4(layer, t["kp"], t.get("vp"), pages(t["table"], BLOCKS), t["first"], t["lens"],
                                                    pages(t["table2"], BLOCKS), t["kw"], t.get("vw")),
                dict(kp=pool, table=table, first=each, lens=each, table2=table, kw=wide, **v(dict(vp=pool, vw=wide))))
    q = (BF16, (N, 4, HD))
    return (lambda t: binding.attn_decode_paged_fp4(layer, t["q"], t["kp"], t.get("vp"), pages(t["table"], BLOCKS), t["lens"], t["out"], t["lse"], ws=t["ws"]),
            dict(q=q, kp=pool, table=table, lens=each, out=q, lse=(F32, (N, 4)), ws=(U8, (4096,)), **v(dict(vp=pool))))


ALL = [("tables", False)] + [(n, e) for n in ("write", "read", "decode") for e in (False, True)]
EACH = [pytest.param(n, e, x, id=f"{n}{'-keqv' if e else ''}-{x}") for n, e in ALL for x in cases(n, e)[1]]


@pytest.mark.parametrize("name,k_eq_v", ALL)
def test_good_tensors_reach_the_library(lib, name, k_eq_v):
    call, want = cases(name, k_eq_v)
    call({x: Tensor(d, *s) for x, (d, s) in want.items()})
    assert lib.calls == 1


@pytest.mark.parametrize("name,k_eq_v,arg", EACH)
def test_one_wrong_tensor(lib, name, k_eq_v, arg):
    """Another type, device or number of dimensions, a row more or less, strides: refused, whichever tensor
    it is (but for what a caller may choose: the length of a list, more table rows, any workspace, how many
    rows k has where there is no v)."""
    call, want = cases(name, k_eq_v)
    dtype, shape = want[arg]
    loose = arg in ("free", "slots", "ws")  # any length
    bad = [Tensor(dtype, *shape, device=1), Tensor(dtype, *shape, device=-1)]
    if arg not in ("pos", "next"):  # (one number has no strides)
        bad.append(Tensor(dtype, *shape, packed=False))
    if arg not in ("table", "table2") or name == "tables":  # (make_pages has looked at the type)
        bad += [Tensor(t, *shape) for t in (I32, F32, BF16, U8, I64, torch.float16) if t != dtype and arg != "ws"]
    else:
        bad.pop()
    if not loose and (name, k_eq_v, arg) != ("write", True, "k"):
        bad.append(Tensor(dtype, shape[0] - 1, *shape[1:]))
        if "table" not in arg:
            bad.append(Tensor(dtype, shape[0] + 1, *shape[1:]))
    if "table" not in arg and arg != "ws":
        bad.append(Tensor(dtype, *shape, 1))
        if not loose:
            bad.append(Tensor(dtype, *shape[:-1], shape[-1] + 1))
    for t in bad:
        with pytest.raises(ValueError):
            call({**{x: Tensor(d, *s) for x, (d, s) in want.items()}, arg: t})
    assert lib.calls == 0


@pytest.mark.parametrize("name", ["write", "read", "decode"])
def test_values_are_there_or_not(lib, name):
    for k_eq_v in (False, True):
        call, want = cases(name, k_eq_v)
        other = cases(name, not k_eq_v)[1]
        good = {x: Tensor(d, *s) for x, (d, s) in want.items()}
        for x in set(want) ^ set(other):
            with pytest.raises(binding.PswError):
                call({k: t for k, t in good.items() if k != x} if x in good else {**good, x: Tensor(other[x][0], *other[x][1])})
    assert lib.calls == 0
