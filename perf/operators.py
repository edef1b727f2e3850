"""Measured cases of the latent-attention operators.

Latent attention keeps one row per token in the pages: a latent vector of L
values (RMS-normalised) and R = 64 rotated key values shared by every head.
The operators:

  write    latent_norm_rope_cache_write(_fp8): RMS-norm of the latent, rotation
           of the shared key part and of the queries' rotary part, cache write
           (bf16 pages, or E4M3 codes with one fp32 scale per row)
  decode   attn_decode_latent(_fp8): absorbed form, one query per sequence over
           its pages: scores q . row over all L + R values, values row[:L]
  expand   latent_kv_expand(_fp8): reads pages back and forms every head's 128
           key and 128 value components, row[:L] W^T
  prefill  attn_prefill_latent: expanded form, a chunk of queries per sequence
           over expanded keys (128 + the shared R) and values (128)

With `own` false, run() computes them in elementary torch operations in fp32.
"""
import math

import numpy as np
import torch

own = False

R, NOPE, V, PAGE = 64, 128, 128, 16
EPS, THETA = 1e-6, 10000.0


def listed():
    return [
        # the new tokens of a decode batch: one per sequence, queries rotated into their absorbed rows
        dict(name="write decode 64", op="write", fp8=False, heads=16, latent=512, n=64, new_lo=1, new_hi=1, past_lo=511, past_hi=4095, lens=1),
        # a chunked-prefill step: 8 chunks of 512 tokens
        dict(name="write chunks 8x512", op="write", fp8=False, heads=16, latent=512, n=8, new_lo=512, new_hi=512, past_lo=0, past_hi=8192, lens=2),
        # ragged long chunks into FP8 pages
        dict(name="write fp8 ragged", op="write", fp8=True, heads=32, latent=512, n=5, new_lo=700, new_hi=2048, past_lo=0, past_hi=16384, lens=3),
        # one short sequence behind a window: latency alone
        dict(name="decode tiny", op="decode", fp8=False, heads=4, latent=256, n=1, len_lo=64, len_hi=64, log=False, window=32, softcap=0.0, lens=4),
        # a decode batch of ordinary context lengths
        dict(name="decode batch 64", op="decode", fp8=False, heads=16, latent=512, n=64, len_lo=512, len_hi=4096, log=False, window=0, softcap=0.0, lens=5),
        # long contexts of very unequal length, many heads
        dict(name="decode long 32", op="decode", fp8=False, heads=32, latent=512, n=32, len_lo=1024, len_hi=32768, log=True, window=0, softcap=0.0, lens=6),
        # the decode batch on FP8 pages, with the logit softcap
        dict(name="decode fp8 batch 64", op="decode", fp8=True, heads=16, latent=512, n=64, len_lo=512, len_hi=4096, log=False, window=0, softcap=50.0, lens=7),
        # few sequences of the longest context on FP8 pages, an odd head count
        dict(name="decode fp8 long 3", op="decode", fp8=True, heads=24, latent=512, n=3, len_lo=40001, len_hi=65536, log=False, window=0, softcap=0.0, lens=8),
        # keys and values of a chunked-prefill step's contexts
        dict(name="expand 8 contexts", op="expand", fp8=False, heads=16, latent=512, n=8, len_lo=512, len_hi=8704, log=False, lens=9),
        # a few odd contexts read back from FP8 pages
        dict(name="expand fp8 odd", op="expand", fp8=True, heads=8, latent=256, n=3, len_lo=77, len_hi=1001, log=True, lens=10),
        # the chunked-prefill step's attention
        dict(name="prefill 8x512", op="prefill", heads=16, n=8, new_lo=512, new_hi=512, past_lo=0, past_hi=8192, window=0, softcap=0.0, lens=11),
        # long ragged chunks after long contexts
        dict(name="prefill 4x2048", op="prefill", heads=16, n=4, new_lo=1800, new_hi=2048, past_lo=2000, past_hi=16384, window=0, softcap=0.0, lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "expand", "prefill", "prefill"])
    case = dict(op=op, heads=_log_int(rng, 1, 64), lens=rng.randrange(1 << 20))
    if op == "write":
        new = _log_int(rng, 1, 2048)
        case.update(fp8=rng.random() < 0.5, latent=rng.choice([256, 512]), n=_log_int(rng, 1, 9000 // (new + 40)), new_lo=max(1, new // 3),
                    new_hi=new, past_lo=0, past_hi=_log_int(rng, 1, 16384))
    elif op == "decode":
        hi = _log_int(rng, 1, 40000)
        n = _log_int(rng, 1, max(1, min(256, 300000 // hi)))
        case.update(fp8=rng.random() < 0.5, latent=rng.choice([256, 512]), n=n, len_lo=max(1, hi // rng.randint(1, 32)), len_hi=hi,
                    log=rng.random() < 0.5, window=0 if rng.random() < 0.7 else _log_int(rng, 1, 2048), softcap=rng.choice([0.0, 0.0, 30.0, 50.0]))
    elif op == "expand":
        hi = _log_int(rng, 1, 8704)
        case.update(fp8=rng.random() < 0.5, latent=rng.choice([256, 512]), n=_log_int(rng, 1, max(1, min(64, 600000 // (hi * case["heads"])))),
                    len_lo=max(1, hi // rng.randint(1, 16)), len_hi=hi, log=rng.random() < 0.5)
    else:
        new, past = _log_int(rng, 1, 2048), _log_int(rng, 1, 16384)
        room = 60_000_000 * 16 // (case["heads"] * new * (new + past))
        case.update(n=_log_int(rng, 1, max(1, min(16, room))), new_lo=max(1, new // 2), new_hi=new, past_lo=0, past_hi=past,
                    window=0 if rng.random() < 0.7 else _log_int(rng, 1, 4096), softcap=rng.choice([0.0, 0.0, 30.0, 50.0]))
    return case


# ------------------------------------------------------------------ lengths and sizes of a case

def _ints(case, lo, hi, key, log=False):
    r = np.random.RandomState((case["lens"] * 7 + key) % (1 << 31))
    if log and hi > lo:
        return np.minimum(hi, np.exp(r.uniform(math.log(lo), math.log(hi + 1), case["n"])).astype(np.int64)).clip(lo)
    return r.randint(lo, hi + 1, case["n"]).astype(np.int64)


def _lengths(case):
    """(new tokens, cached tokens before them) of every sequence."""
    if case["op"] in ("write", "prefill"):
        return _ints(case, case["new_lo"], case["new_hi"], 1), _ints(case, case["past_lo"], case["past_hi"], 2)
    total = _ints(case, case["len_lo"], case["len_hi"], 1, case["log"])
    return np.ones_like(total), total - 1


def _scale(case):
    return 1.0 / math.sqrt(NOPE + R)


def work(case):
    new, past = _lengths(case)
    total, H = new + past, case["heads"]
    if case["op"] == "prefill":
        W = case["window"]
        pairs, keys = 0, 0
        for s, p in zip(new.tolist(), past.tolist()):
            seen = np.arange(p + 1, p + s + 1)
            pairs += int((np.minimum(seen, W) if W else seen).sum())
            keys += min(p + s, W + s - 1) if W else p + s
        rows = int(new.sum())
        return dict(bytes=rows * H * (2 * (NOPE + R) + 2 * V + 4) + keys * (H * 2 * (NOPE + V) + 2 * R), flops=2 * H * pairs * (NOPE + R + V))
    L = case["latent"]
    row = L + R + 4 if case["fp8"] else 2 * (L + R)
    if case["op"] == "write":
        n = int(new.sum())
        return dict(bytes=n * (2 * (L + R) + row + H * R * 4) + 4 * L, flops=n * (6 * L + 4 * R * (H + 1)))
    if case["op"] == "decode":
        seen = int((np.minimum(total, case["window"]) if case["window"] else total).sum())
        return dict(bytes=seen * row + case["n"] * H * (2 * (L + R) + 2 * L + 4), flops=2 * H * seen * (2 * L + R))
    n = int(total.sum())
    return dict(bytes=n * (row + 2 * H * (NOPE + V) + 2 * R) + 2 * H * (NOPE + V) * L, flops=2 * n * L * H * (NOPE + V))


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _rows(g, n, L):
    """n cached rows: a normalised latent and the rotated key part."""
    x = torch.randn((n, L + R), device="cuda", generator=g)
    return x / x[:, :L].square().mean(1, keepdim=True).sqrt()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, past = _lengths(case)
    total, n, H = new + past, case["n"], case["heads"]
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    cu = lambda a: i32(np.concatenate([[0], np.cumsum(a)]))  # noqa: E731
    s = dict(case=case, new=new, total=total, cu_new=cu(new), past_lens=i32(past), seq_lens=i32(total))
    if case["op"] == "prefill":
        nq, nk = int(new.sum()), int(total.sum())
        s.update(cu_k=cu(total), q=_randn(g, nq, H, NOPE + R).bfloat16(), kv=_randn(g, nk, H, NOPE + V).bfloat16(), k_rope=_randn(g, nk, R).bfloat16(),
                 out=torch.empty(nq, H, V, device="cuda", dtype=torch.bfloat16), lse=torch.empty(nq, H, device="cuda"), max_new=int(new.max()))
        s["max_k"] = int(total.max())
        if own:
            from paged_sliding_window_gb300 import binding, workloads
            s["layer"] = workloads.LatentLayer(H, 512, window=case["window"], softcap=case["softcap"], scale=_scale(case))
            s["binding"] = binding
        return s
    L = case["latent"]
    pages = -(-total // PAGE)
    blocks = int(pages.sum()) + 7
    perm = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
    at = np.concatenate([[0], np.cumsum(pages)])
    table = torch.full((n, int(pages.max())), -1, dtype=torch.int32, device="cuda")
    rows = torch.arange(table.shape[1], device="cuda")[None, :]
    first = torch.tensor(at[:-1], device="cuda")[:, None]
    have = rows < torch.tensor(pages, device="cuda")[:, None]
    table[have] = perm[(first + rows)[have]]
    s.update(table=table, blocks=blocks)
    if case["op"] == "write":
        T = int(new.sum())
        s.update(ckv=(2.0 * _randn(g, T, L + R)).bfloat16(), q=_randn(g, T, H, NOPE + R).bfloat16(), weight=1.0 + 0.1 * _randn(g, L),
                 q_abs=torch.zeros(T, H, L + R, device="cuda", dtype=torch.bfloat16))
        if case["fp8"]:
            s.update(pool=torch.zeros(blocks, PAGE, L + R, device="cuda", dtype=torch.uint8), row_scale=torch.zeros(blocks, PAGE, device="cuda"))
        else:
            s.update(pool=torch.zeros(blocks, PAGE, L + R, device="cuda", dtype=torch.bfloat16))
    else:
        x = _rows(g, blocks * PAGE, L)
        if case["fp8"]:
            amax = x.abs().amax(1, keepdim=True)
            s.update(pool=(x * (448.0 / amax)).to(torch.float8_e4m3fn).view(torch.uint8).view(blocks, PAGE, L + R),
                     row_scale=(amax / 448.0).view(blocks, PAGE).contiguous())
        else:
            s.update(pool=x.bfloat16().view(blocks, PAGE, L + R))
        if case["op"] == "decode":
            s.update(q=_randn(g, n, H, L + R).bfloat16(), out=torch.empty(n, H, L, device="cuda", dtype=torch.bfloat16), lse=torch.empty(n, H, device="cuda"))
        else:
            nk = int(total.sum())
            s.update(cu_k=cu(total), w=(_randn(g, H, NOPE + V, L) / math.sqrt(L)).bfloat16(), nk=nk,
                     kv=torch.empty(nk, H, NOPE + V, device="cuda", dtype=torch.bfloat16), k_rope=torch.empty(nk, R, device="cuda", dtype=torch.bfloat16))
    if own:
        from paged_sliding_window_gb300 import binding, workloads
        s["layer"] = workloads.LatentLayer(H, L, window=case.get("window", 0), softcap=case.get("softcap", 0.0), scale=_scale(case))
        s["binding"] = binding
        s["pages"] = binding.make_pages(s["table"], s["blocks"])
        s["norm"] = binding.make_latent_norm(THETA, EPS, s.get("weight"))
        if case["op"] == "decode":
            s["ws"] = binding.alloc_latent_workspace(s["layer"], n)
    return s


# ------------------------------------------------------------------ one pass

def _own_run(s):
    case, b = s["case"], s["binding"]
    if case["op"] == "write":
        L = case["latent"]
        if case["fp8"]:
            b.latent_norm_rope_cache_write_fp8(s["layer"], s["norm"], s["ckv"], s["q"][..., NOPE:], s["cu_new"], s["past_lens"], s["pages"],
                                               s["q_abs"][..., L:], s["pool"], s["row_scale"])
            return dict(pool=s["pool"].view(torch.float8_e4m3fn), scale=s["row_scale"], q=s["q_abs"])
        b.latent_norm_rope_cache_write(s["layer"], s["norm"], s["ckv"], s["q"][..., NOPE:], s["cu_new"], s["past_lens"], s["pages"],
                                       s["q_abs"][..., L:], s["pool"])
        return dict(pool=s["pool"], q=s["q_abs"])
    if case["op"] == "decode":
        if case["fp8"]:
            b.attn_decode_latent_fp8(s["layer"], s["q"], s["pool"], s["row_scale"], s["pages"], s["seq_lens"], s["out"], s["lse"], ws=s["ws"])
        else:
            b.attn_decode_latent(s["layer"], s["q"], s["pool"], s["pages"], s["seq_lens"], s["out"], s["lse"], ws=s["ws"])
        return dict(out=s["out"], lse=s["lse"])
    if case["op"] == "expand":
        if case["fp8"]:
            b.latent_kv_expand_fp8(s["layer"], s["pool"], s["row_scale"], s["pages"], s["cu_k"], s["w"], s["kv"], s["k_rope"])
        else:
            b.latent_kv_expand(s["layer"], s["pool"], s["pages"], s["cu_k"], s["w"], s["kv"], s["k_rope"])
        return dict(kv=s["kv"], k_rope=s["k_rope"])
    b.attn_prefill_latent(s["layer"], s["q"], s["cu_new"], s["past_lens"], s["max_new"], s["kv"], s["k_rope"], s["cu_k"], s["out"], s["lse"])
    return dict(out=s["out"], lse=s["lse"])


def _owners(cu, n):
    """For each of n flat rows: its sequence and its place in it."""
    t = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu.long(), t, right=True) - 1
    return b, t - cu.long()[b]


def _slots(s, b, pos):
    return s["table"][b, pos // PAGE].long() * PAGE + pos % PAGE


def _turn(x, pos):
    """Rotate-half over the last R values of x at positions pos (angles in 64 bits: positions are far)."""
    f = THETA ** (-torch.arange(R // 2, device=x.device, dtype=torch.float64) * 2 / R)
    a = pos.double()[:, None] * f
    c, sn = a.cos().float(), a.sin().float()
    if x.dim() == 3:
        c, sn = c[:, None], sn[:, None]
    lo, hi = x[..., : R // 2], x[..., R // 2:]
    return torch.cat([lo * c - hi * sn, hi * c + lo * sn], -1)


def _pool_rows(s, slots):
    """Rows of the pool in fp32."""
    rows = s["pool"].view(-1, s["pool"].shape[-1])[slots]
    if s["case"]["fp8"]:
        return rows.view(torch.float8_e4m3fn).float() * s["row_scale"].view(-1)[slots][..., None]
    return rows.float()


def _softmax_out(x, hidden, values):
    """softmax over the last axis of x where not hidden, times values; lse; rows with nothing visible give 0 and -inf."""
    x = x.masked_fill(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (x - m).exp()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, values) / torch.where(l == 0, torch.ones_like(l), l)
    return o, (l.log() + m).squeeze(-1)


def _capped(x, case):
    return case["softcap"] * torch.tanh(x / case["softcap"]) if case["softcap"] else x


def run(state):
    s = state
    if own:
        return _own_run(s)
    case = s["case"]
    if case["op"] == "write":
        L = case["latent"]
        b, i = _owners(s["cu_new"], s["ckv"].shape[0])
        pos = s["past_lens"].long()[b] + i
        x = s["ckv"].float()
        c = x[:, :L] * torch.rsqrt(x[:, :L].square().mean(1, keepdim=True) + EPS) * s["weight"]
        row = torch.cat([c, _turn(x[:, L:], pos)], 1)
        s["q_abs"][..., L:] = _turn(s["q"][..., NOPE:].float(), pos).bfloat16()
        slots = _slots(s, b, pos)
        flat = s["pool"].view(-1, L + R)
        if case["fp8"]:
            amax = row.abs().amax(1, keepdim=True)
            flat[slots] = (row * (448.0 / amax)).to(torch.float8_e4m3fn).view(torch.uint8)
            s["row_scale"].view(-1)[slots] = amax[:, 0] / 448.0
            return dict(pool=s["pool"].view(torch.float8_e4m3fn), scale=s["row_scale"], q=s["q_abs"])
        flat[slots] = row.bfloat16()
        return dict(pool=s["pool"], q=s["q_abs"])
    if case["op"] == "decode":
        L, W = case["latent"], case["window"]
        T = s["table"].shape[1] * PAGE
        j = torch.arange(T, device="cuda")[None, :]
        ln = s["seq_lens"].long()[:, None]
        hidden = (j >= ln) | (j < ln - W) if W else j >= ln
        b = torch.arange(case["n"], device="cuda")[:, None]
        slots = torch.where(hidden, torch.zeros_like(j), _slots(s, b, j))
        k = _pool_rows(s, slots).masked_fill(hidden[..., None], 0.0)
        x = _capped(torch.matmul(s["q"].float(), k.transpose(1, 2)) * _scale(case), case)
        o, lse = _softmax_out(x, hidden[:, None, :], k[..., :L])
        return dict(out=o.bfloat16(), lse=lse)
    if case["op"] == "expand":
        L = case["latent"]
        b, pos = _owners(s["cu_k"], s["nk"])
        row = _pool_rows(s, _slots(s, b, pos))
        kv = torch.matmul(row[:, :L], s["w"].float().view(-1, L).t())
        return dict(kv=kv.bfloat16().view(s["kv"].shape), k_rope=row[:, L:].bfloat16())
    W, H = case["window"], case["heads"]
    nq, nk = s["q"].shape[0], s["kv"].shape[0]
    i = torch.arange(s["max_new"], device="cuda")[None, :]
    j = torch.arange(s["max_k"], device="cuda")[None, :]
    qi = (s["cu_new"].long()[:-1, None] + i).clamp(max=nq - 1)
    kj = (s["cu_k"].long()[:-1, None] + j).clamp(max=nk - 1)
    p = (s["past_lens"].long()[:, None] + i)[:, :, None]
    hidden = j[:, None, :] > p
    if W:
        hidden = hidden | (p - j[:, None, :] >= W)
    kv = s["kv"][kj].float().permute(0, 2, 1, 3)
    k = torch.cat([kv[..., :NOPE], s["k_rope"][kj].float()[:, None].expand(-1, H, -1, -1)], -1)
    q = s["q"][qi].float().permute(0, 2, 1, 3)
    x = _capped(torch.matmul(q, k.transpose(2, 3)) * _scale(case), case)
    o, lse = _softmax_out(x, hidden[:, None], kv[..., NOPE:])
    live = i < (s["cu_new"].long()[1:] - s["cu_new"].long()[:-1])[:, None]
    return dict(out=o.permute(0, 2, 1, 3)[live].bfloat16(), lse=lse.permute(0, 2, 1)[live])


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    """Sequence by sequence, unpadded, in float64."""
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    new, total = s["new"].tolist(), s["total"].tolist()
    H, f64 = case["heads"], torch.float64
    seqs = range(case["n"])

    def attend(q, k, v, first_pos):
        """q [H, n, d] at positions first_pos + 0..n-1 over k [H or 1, t, d], v [H or 1, t, e]."""
        x = torch.einsum("hnd,htd->hnt", q, k.expand(H, -1, -1)) * _scale(case)
        if case["softcap"]:
            x = case["softcap"] * torch.tanh(x / case["softcap"])
        p = first_pos + torch.arange(q.shape[1], device="cuda")[:, None]
        j = torch.arange(k.shape[1], device="cuda")[None, :]
        seen = j <= p
        if case["window"]:
            seen &= p - j < case["window"]
        x.masked_fill_(~seen, -math.inf)
        lse = torch.logsumexp(x, -1)
        return torch.einsum("hnt,hte->hne", x.sub_(lse[..., None]).exp_(), v.expand(H, -1, -1)), lse

    if case["op"] == "prefill":
        outs, lses, q0, k0 = [], [], 0, 0
        for b in seqs:
            q = s["q"][q0:q0 + new[b]].to(f64).transpose(0, 1)
            kv = s["kv"][k0:k0 + total[b]].to(f64).transpose(0, 1)
            rope = s["k_rope"][k0:k0 + total[b]].to(f64).expand(H, -1, -1)
            o, l = attend(q, torch.cat([kv[..., :NOPE], rope], -1), kv[..., NOPE:], total[b] - new[b])
            outs.append(o.transpose(0, 1))
            lses.append(l.transpose(0, 1))
            q0, k0 = q0 + new[b], k0 + total[b]
        return dict(out=torch.cat(outs), lse=torch.cat(lses))

    L = case["latent"]

    def places(b, lo, hi):
        pos = torch.arange(lo, hi, device="cuda")
        return s["table"][b].long().gather(0, pos // PAGE) * PAGE + pos % PAGE

    def rows(b):
        at = places(b, 0, total[b])
        if case["fp8"]:
            return s["pool"].view(torch.float8_e4m3fn).view(-1, L + R)[at].to(f64) * s["row_scale"].view(-1, 1)[at].to(f64)
        return s["pool"].view(-1, L + R)[at].to(f64)

    if case["op"] == "decode":
        both = []
        for b in seqs:
            r = rows(b)
            both.append(attend(s["q"][b].to(f64)[:, None], r[None], r[None, :, :L], total[b] - 1))
        return dict(out=torch.stack([o[:, 0] for o, _ in both]), lse=torch.stack([l[:, 0] for _, l in both]))
    if case["op"] == "expand":
        every = torch.cat([rows(b) for b in seqs])
        return dict(kv=torch.einsum("tl,hel->the", every[:, :L], s["w"].to(f64)), k_rope=every[:, L:])

    def rotated(x, pos):
        i = torch.arange(R // 2, device="cuda", dtype=f64)
        turn = torch.polar(torch.ones_like(i), pos.to(f64)[:, None] * torch.exp(-2 * i / R * math.log(THETA)))
        turn = turn.view(turn.shape[0], *[1] * (x.dim() - 2), R // 2)
        z = torch.complex(x[..., : R // 2].contiguous(), x[..., R // 2:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    pool = torch.zeros(s["blocks"] * PAGE, L + R, device="cuda", dtype=f64)
    scale = torch.zeros(s["blocks"] * PAGE, device="cuda", dtype=f64)
    q_abs = torch.zeros(s["q_abs"].shape, device="cuda", dtype=f64)
    t0 = 0
    for b in seqs:
        t = slice(t0, t0 + new[b])
        x = s["ckv"][t].to(f64)
        pos = torch.arange(total[b] - new[b], total[b], device="cuda")
        c = x[:, :L] / (x[:, :L].pow(2).sum(1, keepdim=True) / L + EPS).sqrt() * s["weight"].to(f64)
        y = torch.cat([c, rotated(x[:, L:], pos)], 1)
        q_abs[t, :, L:] = rotated(s["q"][t, :, NOPE:].to(f64), pos)
        at = places(b, total[b] - new[b], total[b])
        if case["fp8"]:
            big = y.abs().amax(1)
            scale[at] = big / 448
            y = (y * (448 / big)[:, None]).float().to(torch.float8_e4m3fn).to(f64)
        pool[at] = y
        t0 += new[b]
    out = dict(pool=pool.view(s["pool"].shape), q=q_abs)
    if case["fp8"]:
        out["scale"] = scale.view(s["row_scale"].shape)
    return out
