"""Measured cases of the 4-bit KV pages: their tables, write, read-back and decode.

A page of one KV head (16 tokens) is one run of 9 * hd bytes: E2M1 codes, one
E4M3 scale for every 16 values of a row; a float per tensor scales all of it.

  tables  block_table_extend: token offsets, lengths, new block-table entries and
          the slot of every new token, from the requests' lengths and a list of
          free pages
  store   kv_cache_write_fp4, then kv_cache_read_fp4 of the rows just written into
          bf16 pages (what the chunk's own prefill runs on)
  read    kv_cache_read_fp4: whole contexts into bf16 pages
  decode  attn_decode_paged_fp4: one query per sequence over its pages

With `own` false, run() computes them in elementary torch operations in fp32.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the E2M1 codes 0..7; bit 3 is the sign


def listed():
    sliding = dict(n_q=16, n_kv=8, hd=256, keqv=False, window=1024, softcap=0.0, scale=1.0, gs=1.0)
    full = dict(n_q=32, n_kv=4, hd=512, keqv=True, window=0, softcap=0.0, scale=1.0, gs=1.0)
    return [
        # the tables of a decode batch's step: one new token per sequence
        dict(name="tables decode 64", op="tables", n=64, chunks=0, new_lo=1, new_hi=1, past_lo=511, past_hi=4095, lens=1),
        # the tables of a mixed step: 256 decoding sequences and four chunks
        dict(name="tables mixed 260", op="tables", n=260, chunks=4, new_lo=2048, new_hi=2048, past_lo=0, past_hi=16384, lens=2),
        # the new tokens of a sliding layer's decode batch
        dict(name="store decode 64", op="store", n_kv=8, hd=256, keqv=False, gs=1.0, n=64, new_lo=1, new_hi=1, past_lo=511, past_hi=4095, lens=9),
        # a chunked-prefill step's rows, stored and read back for the chunk's attention
        dict(name="store chunks 8x512", op="store", n_kv=4, hd=256, keqv=False, gs=1.0, n=8, new_lo=512, new_hi=512, past_lo=0, past_hi=8192, lens=3),
        # ragged long chunks of a full layer whose values are its keys, scaled
        dict(name="store ragged keqv", op="store", n_kv=4, hd=512, keqv=True, gs=0.37, n=5, new_lo=700, new_hi=2048, past_lo=0, past_hi=16384, lens=4),
        # the contexts of a chunked-prefill step read back
        dict(name="read 8 contexts", op="read", n_kv=8, hd=256, keqv=False, gs=1.0, n=8, len_lo=512, len_hi=8704, log=False, window=0, lens=5),
        # what a window leaves of a few odd contexts of a wide layer
        dict(name="read odd windows", op="read", n_kv=3, hd=512, keqv=False, gs=2.5, n=3, len_lo=77, len_hi=1001, log=True, window=200, lens=6),
        # one short sequence behind a window: latency alone
        dict(sliding, name="decode tiny", op="decode", n_q=4, n_kv=2, window=32, n=1, len_lo=64, len_hi=64, log=False, lens=7),
        # a sliding layer's decode batch
        dict(sliding, name="decode sliding 64", op="decode", n=64, len_lo=512, len_hi=4096, log=False, lens=8),
        # a full layer's decode batch of very unequal contexts
        dict(full, name="decode full keqv 32", op="decode", n=32, len_lo=1024, len_hi=32768, log=True, lens=10),
        # few sequences of the longest context, odd head counts, softcap
        dict(sliding, name="decode long 3", op="decode", n_q=21, n_kv=7, window=0, softcap=50.0, scale=0.0625, gs=0.37, n=3, len_lo=40001, len_hi=65536, log=False, lens=11),
        # the decode rows of a mixed step, many of them short
        dict(sliding, name="decode mixed 256", op="decode", n=256, len_lo=16, len_hi=16384, log=True, lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "store", "read", "decode", "decode", "decode"])
    case = dict(op=op, lens=rng.randrange(1 << 20))
    if op == "tables":
        n = _log_int(rng, 1, 1024)
        new = _log_int(rng, 1, 2048)
        case.update(n=n, chunks=rng.randint(0, min(n, max(1, 16000 // new))), new_lo=max(1, new // 3), new_hi=new, past_lo=0, past_hi=_log_int(rng, 1, 16384))
        return case
    case.update(n_kv=_log_int(rng, 1, 8), hd=rng.choice([256, 512]), keqv=rng.random() < 0.3, gs=rng.choice([1.0, 1.0, 0.37, 2.5]))
    per_token = case["n_kv"] * case["hd"]
    if op == "store":
        new = _log_int(rng, 1, 2048)
        case.update(n=_log_int(rng, 1, max(1, min(64, 16_000_000 // (per_token * new)))), new_lo=max(1, new // 3), new_hi=new, past_lo=0, past_hi=_log_int(rng, 1, 16384))
        return case
    hi = _log_int(rng, 1, 40000)
    case.update(len_lo=max(1, hi // rng.randint(1, 32)), len_hi=hi, log=rng.random() < 0.5, window=0 if rng.random() < 0.6 else _log_int(rng, 1, 2048))
    if op == "read":
        case.update(n=_log_int(rng, 1, max(1, min(64, 80_000_000 // (per_token * hi)))))
        return case
    case.update(n_q=case["n_kv"] * _log_int(rng, 1, 12), softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), scale=rng.choice([1.0, 0.0625]))
    case.update(n=_log_int(rng, 1, max(1, min(256, 250_000_000 // (per_token * hi)))))
    return case


# ------------------------------------------------------------------ lengths and sizes of a case

def _ints(case, lo, hi, key, log=False):
    r = np.random.RandomState((case["lens"] * 7 + key) % (1 << 31))
    if log and hi > lo:
        return np.minimum(hi, np.exp(r.uniform(math.log(lo), math.log(hi + 1), case["n"])).astype(np.int64)).clip(lo)
    return r.randint(lo, hi + 1, case["n"]).astype(np.int64)


def _lengths(case):
    """(new tokens, cached tokens before them) of every sequence."""
    if case["op"] in ("tables", "store"):
        new = _ints(case, case["new_lo"], case["new_hi"], 1)
        if case["op"] == "tables":
            new[: case["n"] - case["chunks"]] = 1
        return new, _ints(case, case["past_lo"], case["past_hi"], 2)
    total = _ints(case, case["len_lo"], case["len_hi"], 1, case["log"])
    return np.ones_like(total), total - 1


def _first(case, total):
    """First position wanted of every sequence."""
    return np.maximum(0, total - case["window"]) if case["window"] else np.zeros_like(total)


def _pages(x):
    return -(-x // PAGE)


def work(case):
    new, past = _lengths(case)
    total = new + past
    if case["op"] == "tables":
        added = int((_pages(total) - _pages(past)).sum())
        return dict(bytes=16 * case["n"] + 8 * added + 8 * int(new.sum()), flops=0)
    per = case["n_kv"] * (1 if case["keqv"] else 2)
    packed, wide = per * case["hd"] * 9 // 16, per * case["hd"] * 2
    if case["op"] == "store":
        rows = int(new.sum())
        return dict(bytes=rows * 2 * (packed + wide), flops=rows * per * case["hd"] * 4)
    seen = int((total - _first(case, total)).sum())
    if case["op"] == "read":
        return dict(bytes=seen * (packed + wide), flops=seen * per * case["hd"])
    n, q = case["n"], case["n_q"] * case["hd"]
    return dict(bytes=seen * packed + n * (4 * q + 4 * case["n_q"]), flops=4 * q * seen)


# ------------------------------------------------------------------ the pages

def _places(hd, device):
    """Where a page keeps the byte of values (2 i, 2 i + 1) of token r, [16, hd / 2], and the scale of
    block k (values 16 k .. 16 k + 15), [16, hd / 16]."""
    r = torch.arange(PAGE, device=device)[:, None]
    i = torch.arange(hd // 2, device=device)[None, :]
    unit, part = (i % 128) // 16, i // 128
    codes = part * 2048 + r * 128 + (unit ^ (r & 7)) * 16 + i % 16
    k = torch.arange(hd // 16, device=device)[None, :]
    c, t, e = k // 8, k // 2 % 4, k % 2
    c = c if hd == 256 else c % 2 * 2 + c // 2
    scales = PAGE * hd // 2 + r * (hd // 16) + t * (hd // 64) + c * 2 + e
    return codes, scales


def _quantise(x, gs):
    """Rows x [..., hd] as bytes of two codes [..., hd / 2] and scale bytes [..., hd / 16]."""
    y = (x.float() * float(np.float32(1.0) / np.float32(gs))).clamp(-4096.0, 4096.0).unflatten(-1, (-1, 16))
    s8 = (y.abs().amax(-1) * (1.0 / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    a = (y.abs() / s).nan_to_num(0.0, posinf=0.0)  # nothing is left of a block whose scale is 0
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)) | (torch.signbit(y).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8)


def _values(pages, hd, gs):
    """What pages [..., 9 hd] stand for: fp32 [..., 16, hd]."""
    codes, scales = _places(hd, pages.device)
    level = torch.tensor(LEVELS, device=pages.device)
    level = torch.cat([level, -level])
    byte = torch.arange(256, device=pages.device)
    pair = torch.stack([level[byte & 15], level[byte >> 4]], -1)
    x = pair[pages[..., codes].int()].flatten(-2)
    s = pages[..., scales].view(torch.float8_e4m3fn).float() * gs
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs

def _rows(g, *shape):
    """Head vectors as they leave a layer's norm."""
    x = torch.randn(shape, device="cuda", generator=g)
    return x / x.square().mean(-1, keepdim=True).sqrt()


def _pool(g, case, blocks):
    """A pool of random rows [blocks, n_kv, 9 hd]."""
    hd = case["hd"]
    codes, scales = _places(hd, "cuda")
    pool = torch.empty(blocks, case["n_kv"], 9 * hd, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (case["n_kv"] * PAGE * hd))
    for b in range(0, blocks, step):
        part = pool[b:b + step]
        part[..., codes], part[..., scales] = _quantise(_rows(g, part.shape[0], case["n_kv"], PAGE, hd), case["gs"])
    return pool


def _table(g, pages, width, blocks):
    perm = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
    at = np.concatenate([[0], np.cumsum(pages)])
    table = torch.full((len(pages), width), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")[None, :]
    have = col < torch.tensor(pages, device="cuda")[:, None]
    table[have] = perm[(torch.tensor(at[:-1], device="cuda")[:, None] + col)[have]]
    return table, perm[int(at[-1]):].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, past = _lengths(case)
    total, n = new + past, case["n"]
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=case, new=new, total=total, new_lens=i32(new), past_lens=i32(past), seq_lens=i32(total),
             cu_new=i32(np.concatenate([[0], np.cumsum(new)])))
    blocks = int(_pages(total).sum()) + 7
    width = int(_pages(total).max())
    if case["op"] == "tables":
        before, free = _table(g, _pages(past), width, blocks)
        s.update(table=before, free=free, free_pos=i32([3]), free_next=i32([0]), out_cu=torch.zeros_like(s["cu_new"]), out_lens=torch.zeros_like(s["seq_lens"]),
                 slots=torch.full((int(new.sum()),), -1, dtype=torch.int64, device="cuda"))
    else:
        hd, n_kv = case["hd"], case["n_kv"]
        s.update(table=_table(g, _pages(total), width, blocks)[0], blocks=blocks)
        fill = (lambda: torch.zeros(blocks, n_kv, 9 * hd, dtype=torch.uint8, device="cuda")) if case["op"] == "store" else (lambda: _pool(g, case, blocks))
        s["k_pool"] = fill()
        s["v_pool"] = None if case["keqv"] else fill()
        if case["op"] == "store":
            s["k"] = _rows(g, int(new.sum()), n_kv, hd).bfloat16()
            s["v"] = None if case["keqv"] else _rows(g, int(new.sum()), n_kv, hd).bfloat16()
        if case["op"] in ("store", "read"):  # bf16 pages of their own for the rows wanted
            first = past if case["op"] == "store" else _first(case, total)
            wide = int((_pages(total) - first // PAGE).sum()) + 3
            s["first"], s["rows"] = i32(first), int((total - first).sum())
            s["wide_table"] = torch.full_like(s["table"], -1)
            perm = torch.randperm(wide, device="cuda", generator=g).to(torch.int32)
            col = torch.arange(width, device="cuda")[None, :]
            have = (col >= (s["first"] // PAGE)[:, None]) & (col < torch.tensor(_pages(total), device="cuda")[:, None])
            s["wide_table"][have] = perm[: int(have.sum())]
            s["k_wide"] = torch.zeros(wide, PAGE, n_kv, hd, dtype=torch.bfloat16, device="cuda")
            s["v_wide"] = None if case["keqv"] else torch.zeros_like(s["k_wide"])
        else:
            s.update(q=_rows(g, n, case["n_q"], hd).bfloat16(), out=torch.empty(n, case["n_q"], hd, dtype=torch.bfloat16, device="cuda"),
                     lse=torch.empty(n, case["n_q"], device="cuda"))
    if own:
        from paged_sliding_window_gb300 import binding, workloads
        s["binding"] = binding
        if case["op"] != "tables":
            s["layer"] = workloads.Layer(case.get("n_q", n_kv), n_kv, hd, window=case.get("window", 0), softcap=case.get("softcap", 0.0), scale=case.get("scale", 1.0), k_eq_v=case["keqv"])
            s["pages"] = binding.make_pages(s["table"], blocks)
            if "wide_table" in s:
                s["wide_pages"] = binding.make_pages(s["wide_table"], s["k_wide"].shape[0])
            if "q" in s:
                s["ws"] = binding.alloc_fp4_workspace(s["layer"], n)
    return s


# ------------------------------------------------------------------ one pass

def _own_run(s):
    case, b = s["case"], s["binding"]
    if case["op"] == "tables":
        b.block_table_extend(s["table"], s["past_lens"], s["new_lens"], s["free"], s["free_pos"], s["free_next"], s["out_cu"], s["out_lens"], s["slots"])
        return dict(table=s["table"], cu=s["out_cu"], lens=s["out_lens"], slots=s["slots"], next=s["free_next"])
    gs = dict(k_scale=case["gs"], v_scale=case["gs"])
    if case["op"] == "store":
        b.kv_cache_write_fp4(s["layer"], s["k"], s["v"], s["cu_new"], s["past_lens"], s["pages"], s["k_pool"], s["v_pool"], **gs)
    if case["op"] in ("store", "read"):
        b.kv_cache_read_fp4(s["layer"], s["k_pool"], s["v_pool"], s["pages"], s["first"], s["seq_lens"], s["wide_pages"], s["k_wide"], s["v_wide"], **gs)
        return dict(k=s["k_wide"], v=s["v_wide"])
    b.attn_decode_paged_fp4(s["layer"], s["q"], s["k_pool"], s["v_pool"], s["pages"], s["seq_lens"], s["out"], s["lse"], ws=s["ws"], **gs)
    return dict(out=s["out"], lse=s["lse"])


def _owners(cu, n):
    """For each of n flat rows: its sequence and its place in it."""
    t = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu.long(), t, right=True) - 1
    return b, t - cu.long()[b]


def _write(s, x, pool):
    """Quantises the new rows x into their slots of the pool."""
    hd = x.shape[-1]
    b, i = _owners(s["cu_new"], x.shape[0])
    pos = s["past_lens"].long()[b] + i
    blk, r = s["table"][b, pos // PAGE].long(), pos % PAGE
    codes, scales = _places(hd, x.device)
    byte, s8 = _quantise(x, s["case"]["gs"])
    head = torch.arange(x.shape[1], device=x.device)[None, :, None]
    pool[blk[:, None, None], head, codes[r][:, None, :]] = byte
    pool[blk[:, None, None], head, scales[r][:, None, :]] = s8


def _read(s, pool, wide):
    """Rows [first, seq_len) of every sequence as bf16 into its pages of `wide`."""
    count = s["seq_lens"] - s["first"]
    cu = torch.cat([count.new_zeros(1), count.cumsum(0)])
    b, i = _owners(cu, s["rows"])
    pos = s["first"].long()[b] + i
    page, r = pos // PAGE, pos % PAGE
    hd = wide.shape[-1]
    codes, scales = _places(hd, pool.device)
    x = pool[s["table"][b, page].long()]
    level = torch.tensor(LEVELS, device=pool.device)
    level = torch.cat([level, -level])
    byte = x.gather(2, codes[r][:, None, :].expand(-1, x.shape[1], -1))
    v = torch.stack([level[(byte & 15).int()], level[(byte >> 4).int()]], -1).flatten(-2)
    sc = x.gather(2, scales[r][:, None, :].expand(-1, x.shape[1], -1)).view(torch.float8_e4m3fn).float()
    v = (v.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2) * s["case"]["gs"]
    wide[s["wide_table"][b, page].long(), r] = v.bfloat16()


def run(state):
    s = state
    if own:
        return _own_run(s)
    case = s["case"]
    if case["op"] == "tables":
        past, new = s["past_lens"].long(), s["new_lens"].long()
        total = past + new
        s["out_lens"].copy_(total)
        s["out_cu"][1:] = new.cumsum(0)
        have, need = (past + PAGE - 1) // PAGE, (total + PAGE - 1) // PAGE
        before = (need - have).cumsum(0) - (need - have)
        col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
        at = s["free_pos"].long() + before[:, None] + col - have[:, None]
        fresh = (col >= have[:, None]) & (col < need[:, None])
        s["table"].copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].shape[0] - 1)], s["table"]))
        s["free_next"].copy_(s["free_pos"] + (need - have).sum())
        b, i = _owners(s["out_cu"], s["slots"].shape[0])
        pos = past[b] + i
        s["slots"].copy_(s["table"][b, pos // PAGE].long() * PAGE + pos % PAGE)
        return dict(table=s["table"], cu=s["out_cu"], lens=s["out_lens"], slots=s["slots"], next=s["free_next"])
    if case["op"] == "store":
        _write(s, s["k"], s["k_pool"])
        if not case["keqv"]:
            _write(s, s["v"], s["v_pool"])
    if case["op"] in ("store", "read"):
        _read(s, s["k_pool"], s["k_wide"])
        if not case["keqv"]:
            _read(s, s["v_pool"], s["v_wide"])
        return dict(k=s["k_wide"], v=s["v_wide"])
    # one query per sequence over the pages that its window leaves
    W, n, n_kv, hd = case["window"], case["n"], case["n_kv"], case["hd"]
    ln = s["seq_lens"].long()
    lo = (ln - W).clamp(min=0) if W else torch.zeros_like(ln)
    width = s["table"].shape[1]
    P = min(width, W // PAGE + 2) if W else width
    page = (lo // PAGE)[:, None] + torch.arange(P, device="cuda")
    pos = (page * PAGE)[:, :, None] + torch.arange(PAGE, device="cuda")
    hidden = ((pos < lo[:, None, None]) | (pos >= ln[:, None, None])).flatten(1)
    live = page * PAGE < ln[:, None]
    blk = torch.where(live, s["table"].long().gather(1, page.clamp(max=width - 1)), torch.zeros_like(page))
    k = _values(s["k_pool"][blk], hd, case["gs"]).transpose(1, 2).flatten(2, 3)  # [n, n_kv, P * 16, hd]
    q = s["q"].float().view(n, n_kv, -1, hd)
    x = torch.matmul(q, k.transpose(2, 3)) * case["scale"]
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    x = x.masked_fill(hidden[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    l = p.sum(-1, keepdim=True)
    v = k if case["keqv"] else _values(s["v_pool"][blk], hd, case["gs"]).transpose(1, 2).flatten(2, 3)
    o = torch.matmul(p, v) / l
    return dict(out=o.view(n, -1, hd).bfloat16(), lse=(l.log() + m).view(n, -1))


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """Sequence by sequence, from the definition; nothing of it is a computed number for the tables."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    new, total = s["new"].tolist(), s["total"].tolist()
    f64 = torch.float64
    if case["op"] == "tables":
        table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy()
        at, slots = int(s["free_pos"]), []
        for b in range(case["n"]):
            for p in range(total[b] - new[b], total[b]):
                if p % PAGE == 0:
                    table[b, p // PAGE] = free[at]
                    at += 1
                slots.append(int(table[b, p // PAGE]) * PAGE + p % PAGE)
        t = lambda a, d: torch.tensor(np.asarray(a), dtype=d, device="cuda")  # noqa: E731
        return dict(table=t(table, torch.int32), cu=s["cu_new"], lens=s["seq_lens"], slots=t(slots, torch.int64), next=t([at], torch.int32))
    hd, gs = case["hd"], case["gs"]

    def grid(x):
        """A row in 64 bits, rounded to what its blocks of 16 can hold."""
        y = (x.to(f64) / gs).unflatten(-1, (-1, 16))
        sc = (y.abs().amax(-1, keepdim=True) / 6).clamp(max=448).float().to(torch.float8_e4m3fn).to(f64)
        z = y / torch.where(sc == 0, torch.full_like(sc, math.inf), sc)
        a = z.abs().clamp(max=6.0)
        step = 2.0 ** torch.floor(torch.log2(a.clamp(min=1.0))) / 2  # the distance of neighbours
        return (torch.copysign(torch.round(a / step) * step, z) * sc * gs).flatten(-2)

    def rows(pool, b, lo, hi):
        """Cached rows [lo, hi) of sequence b: [hi - lo, n_kv, hd]."""
        pos = torch.arange(lo, hi, device="cuda")
        page = pool[s["table"][b].long()[pos // PAGE]]
        r, d = (pos % PAGE)[:, None], torch.arange(hd, device="cuda")[None, :]
        u = d % 256 // 32
        byte = page.gather(2, (d // 256 * 2048 + r * 128 + (u ^ (r % 8)) * 16 + d % 32 // 2)[:, None].expand(-1, page.shape[1], -1)).long()
        code = byte >> (4 * (d % 2)) & 15
        e, m = code % 8 // 2, code % 2
        mag = torch.where(e == 0, m.to(f64) / 2, (2.0 ** (e.to(f64) - 1)) * (1 + m.to(f64) / 2))
        k = d // 16
        c = k // 8
        c = c if hd == 256 else torch.tensor([0, 2, 1, 3], device="cuda")[c]
        at = 8 * hd + r * (hd // 16) + k % 8 // 2 * (hd // 64) + c * 2 + k % 2
        sc = page.gather(2, at[:, None].expand(-1, page.shape[1], -1)).view(torch.float8_e4m3fn).to(f64)
        return torch.where(code >= 8, -mag, mag) * sc * gs

    if case["op"] in ("store", "read"):
        outs = {}
        for name in ("k", "v"):
            if s[name + "_pool"] is None:
                outs[name] = None
                continue
            wide, t0 = s[name + "_wide"].to(f64), 0
            for b in range(case["n"]):
                lo = int(s["first"][b])
                x = grid(s[name][t0:t0 + new[b]]) if case["op"] == "store" else rows(s[name + "_pool"], b, lo, total[b])
                pos = torch.arange(lo, total[b], device="cuda")
                wide[s["wide_table"][b].long()[pos // PAGE], pos % PAGE] = x
                t0 += new[b]
            outs[name] = wide
        return outs
    outs, lses = [], []
    for b in range(case["n"]):
        lo = max(0, total[b] - case["window"]) if case["window"] else 0
        k = rows(s["k_pool"], b, lo, total[b])
        v = k if case["keqv"] else rows(s["v_pool"], b, lo, total[b])
        q = s["q"][b].to(f64).view(case["n_kv"], -1, hd)
        x = torch.einsum("hgd,thd->hgt", q, k) * case["scale"]
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        lse = torch.logsumexp(x, -1)
        outs.append(torch.einsum("hgt,thd->hgd", (x - lse[..., None]).exp(), v).flatten(0, 1))
        lses.append(lse.flatten())
    return dict(out=torch.stack(outs), lse=torch.stack(lses))
