"""Serving and training operators around the attention kernels: what is measured of them.

* ``norm_rope``: RMS norm of every query and key head and the rotation by position, one pass;
  ``norm_rope_step`` is a training step of it (forward, then the gradients of q, k and both gains).
* ``append``: the K and V rows of new tokens written into a paged cache, as e4m3 codes with a
  power-of-two scale per (position, K/V head), or as they are into a bf16 cache.
* ``read``: the first positions of every sequence gathered back out of the pages.
* ``decode``: attention of one new token per sequence over the 8-bit paged cache.

``own`` False runs them in elementary torch operations, True through the framework's entry points.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False


DEV = "cuda"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # a serving step's new tokens: 64 sequences, 64 query heads on 8 K/V heads, q and k still inside the packed
        # projection; latency counts
        dict(name="norm_rope token B64", op="norm_rope", dtype="bf16", B=64, N=1, H=64, Hkv=8, d=128, norm=True,
             interleaved=False, packed=True, table=8192, positions="drawn"),
        # a prompt on its way into the forward kernel
        dict(name="norm_rope prompt N4096", op="norm_rope", dtype="bf16", B=1, N=4096, H=64, Hkv=8, d=128, norm=True,
             interleaved=False, packed=True, table=32768, positions="none"),
        # rotation only, adjacent pairs, fp32, odd sizes: inputs of the exact fp32 forward
        dict(name="rope fp32 ragged", op="norm_rope", dtype="fp32", B=3, N=333, H=6, Hkv=3, d=64, norm=False,
             interleaved=True, packed=False, table=1000, positions="padded"),
        # a training step at the long-sequence size
        dict(name="norm_rope step N16384", op="norm_rope_step", dtype="bf16", B=1, N=16384, H=32, Hkv=32, d=128,
             norm=True, interleaved=False, packed=False, table=16384, positions="none", weights="bf16"),
        # a training step on short padded rows, gains kept in fp32
        dict(name="norm_rope step ragged d64", op="norm_rope_step", dtype="bf16", B=4, N=1001, H=16, Hkv=4, d=64,
             norm=True, interleaved=False, packed=False, table=2048, positions="padded", weights="fp32"),
        # one new token of each of 64 sequences into an 8-bit cache
        dict(name="append token B64", op="append", cache="fp8", B=64, N=1, Hkv=8, d=128, page=16, max_start=500,
             ragged=False),
        # eight prompts of different lengths into an 8-bit cache
        dict(name="append prompts B8 N4096", op="append", cache="fp8", B=8, N=4096, Hkv=8, d=128, page=16, max_start=100,
             ragged=True),
        # cached contexts read back for a prompt's next part
        dict(name="read contexts B8", op="read", cache="fp8", B=8, lo=512, hi=8192, Hkv=8, d=128, page=16),
        # one short context out of a bf16 cache
        dict(name="read short bf16", op="read", cache="bf16", B=1, lo=200, hi=200, Hkv=4, d=64, page=8),
        # the decode step of a full batch: 64 sequences of 512 to 8192 positions
        dict(name="decode B64 8192", op="decode", B=64, lo=512, hi=8192, H=64, Hkv=8, d=128, page=16, window=-1),
        # one long conversation alone
        dict(name="decode B1 100000", op="decode", B=1, lo=100000, hi=100000, H=32, Hkv=8, d=128, page=64, window=-1),
        # a short one, every query head with K/V of its own
        dict(name="decode B1 300 d64", op="decode", B=1, lo=300, hi=300, H=16, Hkv=16, d=64, page=16, window=-1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_step", "append", "read", "decode", "decode"])
    d = rng.choice([64, 128])
    Hkv = _log(rng, 1, 16)
    G = _log(rng, 1, 16)
    if op in ("norm_rope", "norm_rope_step"):
        H = Hkv * G
        B = _log(rng, 1, 64)
        # at most about the work of the long training step
        N = _log(rng, 1, max(1, min(16384, (1 << 26) // (B * (H + Hkv) * d))))
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp32"]), B=B, N=N, H=H, Hkv=Hkv, d=d,
                 norm=rng.random() < 0.75, interleaved=rng.random() < 0.4, packed=rng.random() < 0.5,
                 table=N + rng.randrange(0, 5000), positions=rng.choice(["none", "drawn", "padded"]))
        if op == "norm_rope_step":
            c["norm"] = True
            c["weights"] = rng.choice(["bf16", "fp32"]) if c["dtype"] == "bf16" else "fp32"
        return c
    page = rng.choice([8, 16, 16, 32, 64, 256])
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(op=op, cache=rng.choice(["fp8", "fp8", "bf16"]), B=B, N=_log(rng, 1, max(1, 32768 // B)), Hkv=Hkv,
                    d=d, page=page, max_start=_log(rng, 1, 1000), ragged=rng.random() < 0.5)
    if op == "read":
        B = _log(rng, 1, 32)
        hi = _log(rng, 1, max(1, 32768 // B))
        return dict(op=op, cache=rng.choice(["fp8", "fp8", "bf16"]), B=B, lo=rng.randrange(0, hi + 1), hi=hi, Hkv=Hkv,
                    d=d, page=page)
    B = _log(rng, 1, 64)
    hi = _log(rng, 1, max(1, min(120000, (1 << 21) // (B * Hkv))))
    return dict(op=op, B=B, lo=rng.randrange(0, hi + 1), hi=hi, H=Hkv * G, Hkv=Hkv, d=d, page=page,
                window=rng.choice([-1, -1, -1, _log(rng, 1, 4096)]))


# --------------------------------------------------------------------------
# what a program has in hand before the call
# --------------------------------------------------------------------------
def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _lengths(case, seed):
    g = torch.Generator(device="cpu").manual_seed(int(seed) + 7)
    return torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=g, dtype=torch.int64)


def _pages(need, page, longest, seed, room=False):
    """A pool with two spare pages (``room``: pages for every sequence's longest state), handed out to the sequences in
    a shuffled order; (pages in the pool, block table).  A row of the table has room for ``longest`` positions, -1 past
    the sequence's last page."""
    g = torch.Generator(device="cpu").manual_seed(int(seed) + 9)
    n = [(int(x) + page - 1) // page for x in need]
    total = (len(n) * ((longest + page - 1) // page) if room else sum(n)) + 2
    order = torch.randperm(total, generator=g, dtype=torch.int64).to(torch.int32)
    table = torch.full((len(n), max(1, (longest + page - 1) // page)), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(n):
        table[b, :k] = order[at:at + k]
        at += k
    return total, table.to(DEV)


def _scale_bytes(x):
    """The 8-bit scale 2^(byte - 127) of rows ``x`` [..., d]: the smallest power of two (not under 2^-126) that brings
    the row's largest magnitude to 448 at most."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)                                  # amax = m 2^e, m in [1/2, 1)
    e = e - 9 + (m > 0.875)                                   # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    return torch.where(torch.isfinite(amax), e + 127, torch.full_like(e, 255)).to(torch.uint8)


def _scale_values(b):
    v = torch.ldexp(torch.ones_like(b, dtype=torch.float32), b.to(torch.int32) - 127)
    return torch.where(b == 255, torch.full_like(v, float("nan")), v)


def _pool8(pages, page, Hkv, d, gen):
    """An 8-bit pool filled by earlier steps: codes [pages, page, Hkv, d] and their scales [pages, Hkv, page]."""
    x = torch.randn((pages, page, Hkv, d), generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn((pages, page, Hkv, 1), generator=gen, device=DEV))
    b = _scale_bytes(x)
    codes = torch.ldexp(x, 127 - b.to(torch.int32).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes, b.permute(0, 2, 1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    s = {"case": dict(case)}
    if op in ("norm_rope", "norm_rope_step"):
        B, N, H, T = case["B"], case["N"], case["H"], case["table"]
        dt = _dtype(case["dtype"])
        if case["packed"]:
            qkv = (1.5 * torch.randn((B, N, H + 2 * Hkv, d), generator=gen, device=DEV)).to(dt)
            s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
        else:
            s["q"] = (1.5 * torch.randn((B, N, H, d), generator=gen, device=DEV)).to(dt)
            s["k"] = (1.5 * torch.randn((B, N, Hkv, d), generator=gen, device=DEV)).to(dt)
        freq = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
        angle = torch.arange(T, dtype=torch.float64, device=DEV)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        if case["positions"] == "none":
            s["pos"] = None
        elif case["positions"] == "drawn":
            s["pos"] = torch.randint(0, T, (B, N), generator=gen, device=DEV, dtype=torch.int32)
        else:  # rows of different lengths, the rest padding
            keep = torch.randint(0, N + 1, (B, 1), generator=gen, device=DEV)
            at = torch.arange(N, device=DEV)[None].expand(B, N)
            s["pos"] = torch.where(at < keep, at, torch.full_like(at, -1)).to(torch.int32)
        s["wq"] = s["wk"] = None
        if case["norm"]:
            wd = _dtype(case.get("weights", case["dtype"]))
            s["wq"], s["wk"] = ((1 + 0.2 * torch.randn((d,), generator=gen, device=DEV)).to(wd) for _ in range(2))
        if op == "norm_rope_step":
            s["gq"] = torch.randn((B, N, H, d), generator=gen, device=DEV).to(dt)
            s["gk"] = torch.randn((B, N, Hkv, d), generator=gen, device=DEV).to(dt)
            for n in ("q", "k", "wq", "wk"):
                s[n] = s[n].detach().requires_grad_(True)
        return s
    page = case["page"]
    if op == "append":
        B, N = case["B"], case["N"]
        g = torch.Generator(device="cpu").manual_seed(int(seed) + 3)
        start = torch.randint(0, case["max_start"] + 1, (B,), generator=g, dtype=torch.int64)
        count = torch.randint(0, N + 1, (B,), generator=g, dtype=torch.int64) if case["ragged"] else torch.full((B,), N)
        pages, s["table"] = _pages((start + count).tolist(), page, case["max_start"] + N, seed, room=True)
        s["start"], s["count"] = start.to(torch.int32).to(DEV), count.to(torch.int32).to(DEV) if case["ragged"] else None
        k = torch.randn((B, N, Hkv, d), generator=gen, device=DEV)
        v = torch.randn((B, N, Hkv, d), generator=gen, device=DEV)
        k *= torch.exp(torch.randn((B, N, Hkv, 1), generator=gen, device=DEV))
        s["k"], s["v"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    else:
        lens = _lengths(case, seed)
        pages, s["table"] = _pages(lens.tolist(), page, case["hi"], seed)
        s["lens"] = lens.to(torch.int32).to(DEV)
        B = case["B"]
    if op == "decode" or case["cache"] == "fp8":
        s["kc"], kb = _pool8(pages, page, Hkv, d, gen)
        s["vc"], vb = _pool8(pages, page, Hkv, d, gen)
        s["sc"] = torch.stack([kb, vb], dim=2).contiguous()       # [pages, Hkv, 2, page]
    else:
        s["kc"] = torch.randn((pages, page, Hkv, d), generator=gen, device=DEV).to(torch.bfloat16)
        s["vc"] = torch.randn((pages, page, Hkv, d), generator=gen, device=DEV).to(torch.bfloat16)
        s["sc"] = None
    if op == "decode":
        s["q"] = torch.randn((B, case["H"], d), generator=gen, device=DEV).to(torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(d)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import exact_io_aware_51_b200 as fa

        return {"norm_rope": _own_norm_rope, "norm_rope_step": _own_step, "append": _own_append, "read": _own_read,
                "decode": _own_decode}[op](fa, s)
    with torch.no_grad():
        return {"norm_rope": _plain_norm_rope, "norm_rope_step": _plain_step, "append": _plain_append,
                "read": _plain_read, "decode": _plain_decode}[op](s)


def _own_norm_rope(fa, s):
    return fa.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], q_weight=s["wq"], k_weight=s["wk"], positions=s["pos"],
                           interleaved=s["case"]["interleaved"])


def _own_step(fa, s):
    q, k = _own_norm_rope(fa, s)
    grads = torch.autograd.grad((q, k), (s["q"], s["k"], s["wq"], s["wk"]), (s["gq"], s["gk"]))
    return (q.detach(), k.detach(), *grads)


def _own_append(fa, s):
    fa.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["start"], kv_scale=s["sc"], count=s["count"])
    return _append_outputs(s)


def _own_read(fa, s):
    return fa.cache_read(s["kc"], s["vc"], s["table"], s["lens"], s["case"]["hi"], kv_scale=s["sc"])


def _own_decode(fa, s):
    w = s["case"]["window"]
    return fa.decode_paged_fp8(s["q"], s["kc"], s["vc"], s["sc"], s["table"], s["lens"], scale=s["scale"],
                               window_left=None if w < 0 else w)


def _append_outputs(s):
    return (s["kc"], s["vc"]) if s["sc"] is None else (s["kc"], s["vc"], s["sc"])


def _pairs(x, interleaved):
    return (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, dim=-1)


def _unpairs(a, b, interleaved):
    return torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)


def _angles(s, N):
    """cos, sin [.., N, 1, d/2] of every row and the rows that are no padding."""
    if s["pos"] is None:
        return s["cos"][:N, None], s["sin"][:N, None], None
    p = s["pos"].clamp(min=0).long()
    return s["cos"][p].unsqueeze(2), s["sin"][p].unsqueeze(2), (s["pos"] >= 0)[..., None, None]


def _plain_rotate(s, x, w):
    inter = s["case"]["interleaved"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    c, sn, keep = _angles(s, x.shape[1])
    a, b = _pairs(y, inter)
    y = _unpairs(a * c - b * sn, b * c + a * sn, inter)
    if keep is not None:
        y = torch.where(keep, y, torch.zeros_like(y))
    return y.to(x.dtype)


def _plain_norm_rope(s):
    return _plain_rotate(s, s["q"], s["wq"]), _plain_rotate(s, s["k"], s["wk"])


def _plain_grad(s, x, w, g):
    inter = s["case"]["interleaved"]
    c, sn, keep = _angles(s, x.shape[1])
    g = g.float()
    if keep is not None:
        g = torch.where(keep, g, torch.zeros_like(g))
    a, b = _pairs(g, inter)
    gr = _unpairs(a * c + b * sn, b * c - a * sn, inter)      # the rotation's transpose
    xf = x.float()
    r = torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-6)
    n = xf * r
    gn = gr * w.float()
    dx = r * (gn - n * (gn * n).mean(-1, keepdim=True))
    dw = (gr * n).sum((0, 1, 2), dtype=torch.float64)
    return dx.to(x.dtype), dw.to(w.dtype)


def _plain_step(s):
    q, k = _plain_norm_rope(s)
    dq, dwq = _plain_grad(s, s["q"], s["wq"], s["gq"])
    dk, dwk = _plain_grad(s, s["k"], s["wk"], s["gk"])
    return q, k, dq, dk, dwq, dwk


def _plain_append(s):
    B, N = s["k"].shape[:2]
    page = s["case"]["page"]
    i = torch.arange(N, device=DEV)[None]
    pos = s["start"].long()[:, None] + i
    keep = (i < s["count"][:, None]) if s["count"] is not None else torch.ones_like(pos, dtype=torch.bool)
    b = torch.arange(B, device=DEV)[:, None].expand(B, N)[keep]
    pos = pos[keep]
    pg, slot = s["table"][b, pos // page].long(), pos % page
    for x, pool, which in ((s["k"], s["kc"], 0), (s["v"], s["vc"], 1)):
        rows = x[keep]                                            # [tokens, Hkv, d]
        if s["sc"] is None:
            pool[pg, slot] = rows
            continue
        y = rows.float()
        sb = _scale_bytes(y)
        codes = torch.ldexp(y, 127 - sb.to(torch.int32).unsqueeze(-1)).to(torch.float8_e4m3fn)
        pool.view(torch.uint8)[pg, slot] = codes.view(torch.uint8)
        s["sc"][pg, :, which, slot] = sb
    return _append_outputs(s)


def _gathered(s, N):
    """The first N positions of every sequence as fp32 K, V [B, N, Hkv, d] (zero past a sequence's end)."""
    page = s["case"]["page"]
    pos = torch.arange(N, device=DEV)
    keep = pos[None] < s["lens"][:, None]
    pg = torch.where(keep, s["table"][:, pos // page], 0).long()
    slot = (pos % page)[None].expand_as(pg)
    out = []
    for pool, which in ((s["kc"], 0), (s["vc"], 1)):
        if s["sc"] is None:
            x = pool[pg, slot].float()
        else:
            x = pool.view(torch.uint8)[pg, slot].view(torch.float8_e4m3fn).float()
            x = x * _scale_values(s["sc"][pg, :, which, slot]).unsqueeze(-1)
        out.append(torch.where(keep[..., None, None], x, torch.zeros_like(x)))
    return out


def _plain_read(s):
    k, v = _gathered(s, s["case"]["hi"])
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_decode(s):
    c = s["case"]
    B, H, d = s["q"].shape
    N, Hkv = c["hi"], c["Hkv"]
    k, v = _gathered(s, N)                                        # [B, N, Hkv, d]
    q = s["q"].float().view(B, Hkv, H // Hkv, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]       # [B, Hkv, G, N]
    pos = torch.arange(N, device=DEV)[None]
    L = s["lens"][:, None]
    seen = pos < L
    if c["window"] >= 0:
        seen = seen & (pos >= L - 1 - c["window"])
    x = torch.where(seen[:, None, None], x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(x - m0)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m0 + torch.log(l), torch.full_like(l, -math.inf))
    return o.reshape(B, H, d).to(torch.bfloat16), lse.reshape(B, H)


# --------------------------------------------------------------------------
# the cost that nothing can avoid
# --------------------------------------------------------------------------
def work(case):
    op, d, Hkv, B = case["op"], case["d"], case["Hkv"], case["B"]
    if op in ("norm_rope", "norm_rope_step"):
        e = 2 if case["dtype"] == "bf16" else 4
        n = B * case["N"] * (case["H"] + Hkv) * d
        angles = min(case["table"], B * case["N"]) * d * 4
        ops = n * (8 if case["norm"] else 3)
        if op == "norm_rope":
            return {"bytes": 2 * n * e + angles, "flops": ops}
        # the step reads q, k and the two gradients once and writes both outputs and both input gradients
        return {"bytes": 6 * n * e + angles, "flops": ops + 16 * n}
    if op == "append":
        n = B * case["N"] * Hkv // (2 if case["ragged"] else 1)
        row = d + 1 if case["cache"] == "fp8" else 2 * d
        return {"bytes": 2 * n * (2 * d + row), "flops": 4 * n * d}
    mean = (case["lo"] + case["hi"]) / 2
    if op == "read":
        row = d + 1 if case["cache"] == "fp8" else 2 * d
        return {"bytes": 2 * B * Hkv * (mean * row + case["hi"] * 2 * d), "flops": 2 * B * Hkv * mean * d}
    if case["window"] >= 0:
        mean = min(mean, case["window"] + 1)
    H = case["H"]
    return {"bytes": 2 * B * Hkv * mean * (d + 1) + 4 * B * H * d + 4 * B * H, "flops": 4 * B * H * mean * d}


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm_rope": _exact_norm_rope, "norm_rope_step": _exact_step, "append": _exact_append,
                "read": _exact_read, "decode": _exact_decode}[case["op"]](s)


def _rotation(s, x):
    """For every row and pair the angle's complex number (from the tables that the call reads), 0 for padding."""
    B, N = x.shape[:2]
    z = torch.complex(s["cos"].double(), s["sin"].double())
    if s["pos"] is None:
        return z[:N].reshape(1, N, 1, -1).expand(B, N, 1, -1)
    z = torch.cat((z, torch.zeros_like(z[:1])))                   # row -1: padding
    return z[s["pos"].long()].reshape(B, N, 1, -1)


def _as_complex(x, inter):
    h = x.shape[-1] // 2
    y = x.reshape(*x.shape[:-1], h, 2) if inter else x.reshape(*x.shape[:-1], 2, h).transpose(-1, -2)
    return torch.view_as_complex(y.contiguous())


def _as_real(z, inter):
    y = torch.view_as_real(z)
    return (y if inter else y.transpose(-1, -2)).reshape(*z.shape[:-1], 2 * z.shape[-1])


def _exact_rows(s, x, w):
    inter = s["case"]["interleaved"]
    x = x.double()
    if w is not None:
        x = w.double() * x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt()
    return _as_real(_as_complex(x, inter) * _rotation(s, x), inter)


def _exact_norm_rope(s):
    return _exact_rows(s, s["q"], s["wq"]), _exact_rows(s, s["k"], s["wk"])


def _exact_step(s):
    out = [_exact_rows(s, s["q"], s["wq"]), _exact_rows(s, s["k"], s["wk"])]
    inter = s["case"]["interleaved"]
    dws = []
    for x, w, g in ((s["q"], s["wq"], s["gq"]), (s["k"], s["wk"], s["gk"])):
        x, w, g = x.double(), w.double(), g.double()
        back = _as_real(_as_complex(g, inter) * _rotation(s, x).conj(), inter)
        ms = (x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6
        dot = (back * w * x).sum(-1, keepdim=True)
        out.append(back * w / ms.sqrt() - x * dot / (x.shape[-1] * ms * ms.sqrt()))
        dws.append((back * x / ms.sqrt()).flatten(0, 2).sum(0))
    return (*out, *dws)


def _e4m3(x):
    """x in 64 bits rounded to the nearest e4m3 value (ties to even)."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _exact_append(s):
    c = s["case"]
    if s["sc"] is None:
        pools = [s["kc"].double(), s["vc"].double()]
    else:
        pools = [s["kc"].float().double(), s["vc"].float().double()]
        sc = s["sc"].clone()
    start, table = s["start"].tolist(), s["table"].tolist()
    count = s["count"].tolist() if s["count"] is not None else [c["N"]] * c["B"]
    for b in range(c["B"]):
        at = torch.arange(start[b], start[b] + count[b])
        pg = torch.tensor(table[b])[at // c["page"]].to(DEV)
        slot = (at % c["page"]).to(DEV)
        for which, x in enumerate((s["k"], s["v"])):
            rows = x[b, :count[b]].double()
            if s["sc"] is None:
                pools[which][pg, slot] = rows
                continue
            amax = rows.abs().amax(-1).cpu().numpy()
            e = np.maximum(np.ceil(np.log2(np.maximum(amax, 1e-300) / 448.0)), -126)
            e = np.where(np.ldexp(448.0, (e - 1).astype(np.int64)) >= amax, np.maximum(e - 1, -126), e)  # log2 near a border
            e = torch.from_numpy(e).to(DEV)
            pools[which][pg, slot] = _e4m3(rows * torch.exp2(-e).unsqueeze(-1))
            sc[pg, :, which, slot] = (e + 127).to(torch.uint8)
    return pools if s["sc"] is None else (*pools, sc)


def _exact_pages(s, b, n):
    """K, V [n, Hkv, d] of one sequence in 64 bits."""
    page = s["case"]["page"]
    k = (n + page - 1) // page
    pg = s["table"][b, :k].long()
    out = []
    for which, pool in enumerate((s["kc"], s["vc"])):
        x = pool.view(torch.uint8)[pg].view(pool.dtype).double() if s["sc"] is not None else pool[pg].double()
        if s["sc"] is not None:
            x = x * torch.exp2(s["sc"][pg, :, which].double() - 127).transpose(1, 2).unsqueeze(-1)
        out.append(x.flatten(0, 1)[:n])
    return out


def _exact_read(s):
    c = s["case"]
    k = torch.zeros((c["B"], c["hi"], c["Hkv"], c["d"]), dtype=torch.float64, device=DEV)
    v = torch.zeros_like(k)
    for b, n in enumerate(s["lens"].tolist()):
        k[b, :n], v[b, :n] = _exact_pages(s, b, n)
    return k, v


def _exact_decode(s):
    c = s["case"]
    B, H, d = s["q"].shape
    o = torch.zeros((B, H, d), dtype=torch.float64, device=DEV)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        k, v = _exact_pages(s, b, n)
        if c["window"] >= 0:
            k, v = k[max(0, n - 1 - c["window"]):], v[max(0, n - 1 - c["window"]):]
        if k.shape[0] == 0:
            continue
        q = s["q"][b].double().view(c["Hkv"], -1, d)
        x = torch.einsum("hgd,nhd->hgn", q, k) * s["scale"]
        lse[b] = torch.logsumexp(x, -1).flatten()
        o[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).reshape(H, d)
    return o, lse
