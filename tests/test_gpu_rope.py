"""Norm and rotation of query and key heads: the CUDA kernels against the fp64 oracle.

Tolerances.  An output is rounded once, by at most half a step (bf16 2^-8, fp32
2^-24 of it).  Before that everything is fp32.  Forward: out = r (x1 (c w1) - x2 (s w2)):
one rounding for each folded coefficient, two for the two-term sum, one for the
product with r; r itself carries half of the relative error of the mean of squares
(at most 8 + 1 + 3 summation steps and the added eps) and two units of rsqrt, 4 *
2^-24.  Together under 16 * 2^-24 = 2^-20 of |x1 c w1| + |x2 s w2| times r.  Backward:
the rotation (3), the gain (1), r (11), the d-term sum of w gr x (16 steps), r^3 and
two products: under 64 * 2^-24 = 2^-18 of r |w| |gr| + |x| r^3 / d sum |w gr x|, with gr
taken in magnitudes.  dw sums `rows` terms, each with at most 32 roundings: (rows +
64) * 2^-24 of the sum of magnitudes.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_51_b200 as fa
import oracle
from oracle import serving as S
from tests.helpers import need_gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 1e-37


def _f(t):
    return t.detach().cpu().double().numpy()


def _case(dtype, B, N, H, Hkv, d, norm, inter, packed, positions, wdtype, seed, rows=None):
    g = torch.Generator().manual_seed(seed)
    rows = rows or N + 5
    if packed:
        x = torch.randn((B, N, H + 2 * Hkv, d), generator=g).to(dtype).cuda()
        q, k = x[:, :, :H], x[:, :, H:H + Hkv]
    else:
        q, k = (torch.randn((B, N, h, d), generator=g).to(dtype).cuda() for h in (H, Hkv))
    ang = torch.rand((rows, d // 2), generator=g, dtype=torch.float64) * 6.3
    cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()
    w = [None, None]
    if norm:
        w = [(1 + 0.3 * torch.randn(d, generator=g)).to(wdtype).cuda() for _ in range(2)]
    pos = None
    if positions:
        pos = torch.randint(-2, rows, (B, N), generator=g, dtype=torch.int32).cuda()
    gq, gk = (torch.randn((B, N, h, d), generator=g).to(dtype).cuda() for h in (H, Hkv))
    return q, k, cos, sin, w, pos, gq, gk


BF, F32 = torch.bfloat16, torch.float32
CASES = [
    # dtype, B, N, H, Hkv, d, norm, interleaved, packed, positions, gains
    (BF, 1, 1, 1, 1, 64, True, False, False, False, BF),
    (BF, 3, 1, 32, 8, 128, True, False, True, True, BF),
    (BF, 2, 37, 5, 3, 128, True, True, True, True, F32),
    (BF, 1, 130, 9, 1, 64, True, False, False, False, F32),
    (BF, 2, 65, 17, 2, 64, False, True, True, False, BF),
    (BF, 1, 200, 64, 8, 128, True, False, True, False, BF),
    (F32, 2, 33, 4, 4, 64, True, True, False, True, F32),
    (F32, 1, 50, 7, 2, 128, True, False, True, True, F32),
    (F32, 3, 21, 6, 3, 128, False, False, False, True, F32),
    (BF, 2, 19, 0, 3, 64, True, False, False, True, BF),       # keys alone
    (F32, 2, 19, 3, 3, 64, True, False, False, True, BF),      # gains in fewer bits than the rows
    (F32, 2, 23, 5, 1, 128, True, True, True, True, BF),
    (F32, 1, 41, 9, 3, 128, False, True, False, False, F32),
]


def _name(c):
    return "-".join(str(x).replace("torch.", "") for x in c)


def _magnitude(y, inter):
    """|first| + |second| of every pair, for both of its features."""
    z = S._pairs(np.abs(y), inter)
    m = z.real + z.imag
    return S._from_pairs(m + 1j * m, inter)


def _check_fwd(x, w, cos, sin, pos, inter, out):
    ref = S.norm_rope(_f(x), None if w is None else _f(w), _f(cos), _f(sin), None if pos is None else pos.cpu().numpy(),
                      1e-6, inter)
    one = np.ones_like(_f(cos)), np.zeros_like(_f(cos))
    mag = _magnitude(S.norm_rope(_f(x), None if w is None else _f(w), *one, None, 1e-6, inter), inter)
    err = np.abs(_f(out) - ref)
    assert np.all(err <= HALF[out.dtype] * np.abs(ref) + 2.0 ** -20 * mag + TINY)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=_name)
def test_forward_matches_oracle(case):
    need_gpu()
    inter = case[7]
    q, k, cos, sin, w, pos, _, _ = _case(*case, seed=11)
    qo, ko = fa.qk_norm_rope_fwd(q, k, cos, sin, w[0], w[1], pos, interleaved=inter)
    _check_fwd(q, w[0], cos, sin, pos, inter, qo)
    _check_fwd(k, w[1], cos, sin, pos, inter, ko)
    assert fa.last_device_status()[0] == 0
    again = fa.qk_norm_rope(q, k, cos, sin, w[0], w[1], pos, interleaved=inter)
    assert torch.equal(again[0], qo) and torch.equal(again[1], ko)


def _check_bwd(x, w, cos, sin, pos, inter, g, dx, dw):
    p = None if pos is None else pos.cpu().numpy()
    X, G, W = _f(x), _f(g), None if w is None else _f(w)
    rx, rw = S.norm_rope_backward(X, W, _f(cos), _f(sin), G, p, 1e-6, inter)
    gr = _magnitude(G, inter)
    if p is not None:
        gr = gr * (p >= 0)[:, :, None, None]
    if W is None:
        mag = gr
    else:
        r = 1 / np.sqrt(np.mean(X * X, axis=-1, keepdims=True) + 1e-6)
        mag = r * np.abs(W) * gr + np.abs(X) * r ** 3 / X.shape[-1] * np.sum(np.abs(W * X) * gr, axis=-1, keepdims=True)
        rows = X[..., 0].size
        wmag = np.sum(gr * np.abs(X) * r, axis=(0, 1, 2))
        assert dw.dtype == w.dtype
        assert np.all(np.abs(_f(dw) - rw) <= HALF[dw.dtype] * np.abs(rw) + (rows + 64) * 2.0 ** -24 * wmag + TINY)
    assert np.all(np.abs(_f(dx) - rx) <= HALF[dx.dtype] * np.abs(rx) + 2.0 ** -18 * mag + TINY)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=_name)
def test_backward_matches_oracle(case):
    need_gpu()
    inter = case[7]
    q, k, cos, sin, w, pos, gq, gk = _case(*case, seed=12)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos, interleaved=inter)
    if case[3]:
        _check_bwd(q, w[0], cos, sin, pos, inter, gq, dq, dwq)
    _check_bwd(k, w[1], cos, sin, pos, inter, gk, dk, dwk)
    again = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos, interleaved=inter)
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert (a is None and b is None) or torch.equal(a, b)  # the sums have one order


@pytest.mark.gpu
def test_backward_of_many_rows_uses_every_block():
    """More (position, head) units than the backward has warps: each walks several."""
    need_gpu()
    case = (BF, 2, 3001, 8, 4, 64, True, False, False, True, F32)
    q, k, cos, sin, w, pos, gq, gk = _case(*case, seed=13)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos)
    _check_bwd(q, w[0], cos, sin, pos, False, gq, dq, dwq)
    _check_bwd(k, w[1], cos, sin, pos, False, gk, dk, dwk)
    qo, ko = fa.qk_norm_rope(q, k, cos, sin, w[0], w[1], pos)
    _check_fwd(q, w[0], cos, sin, pos, False, qo)
    _check_fwd(k, w[1], cos, sin, pos, False, ko)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,inter,d,norm", [(BF, False, 128, True), (BF, True, 64, True), (F32, False, 128, True),
                                                (BF, False, 64, False)])
def test_many_positions_and_heads(dtype, inter, d, norm):
    """Enough warps that each takes eight groups of rows, with heads that do not fill the last group, q out of
    a packed projection."""
    need_gpu()
    rows = 512 // d
    case = (dtype, 1, 3301, 8 * rows + 1, rows + 1, d, norm, inter, True, True, F32)
    q, k, cos, sin, w, pos, gq, gk = _case(*case, seed=23)
    qo, ko = fa.qk_norm_rope(q, k, cos, sin, w[0], w[1], pos, interleaved=inter)
    _check_fwd(q, w[0], cos, sin, pos, inter, qo)
    _check_fwd(k, w[1], cos, sin, pos, inter, ko)
    dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos, interleaved=inter)
    _check_bwd(q, w[0], cos, sin, pos, inter, gq, dq, dwq)
    _check_bwd(k, w[1], cos, sin, pos, inter, gk, dk, dwk)


@pytest.mark.gpu
def test_tensors_beyond_32_bit_offsets():
    """q and its output of 2.3e9 elements: the last positions are those of a small call."""
    need_gpu()
    N, H, d, last = 280000, 64, 128, 37
    g = torch.Generator().manual_seed(24)
    tail = torch.randn((1, last, H, d), generator=g).to(BF).cuda()
    k = torch.randn((1, last, 1, d), generator=g).to(BF).cuda()
    cos, sin = fa.rope_tables(N, d)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(BF).cuda()
    q = torch.zeros((1, N, H, d), dtype=BF, device="cuda")
    kk = torch.zeros((1, N, 1, d), dtype=BF, device="cuda")
    assert q.numel() > 2 ** 31
    q[:, -last:], kk[:, -last:] = tail, k
    pos = torch.arange(N - last, N, dtype=torch.int32, device="cuda").view(1, last)
    want = fa.qk_norm_rope(tail, k, cos, sin, w, w, pos)
    got = fa.qk_norm_rope(q, kk, cos, sin, w, w)
    assert torch.equal(got[0][:, -last:], want[0]) and torch.equal(got[1][:, -last:], want[1])
    assert torch.count_nonzero(got[0][:, :-last]) == 0
    want = fa.qk_norm_rope_bwd(tail, k, cos, sin, tail, k, w, w, pos)
    got = fa.qk_norm_rope_bwd(q, kk, cos, sin, q, kk, w, w)
    assert torch.equal(got[0][:, -last:], want[0]) and torch.equal(got[1][:, -last:], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,H,Hkv,d,N", [(BF, 33, 7, 128, 20001), (BF, 4, 1, 64, 40009), (F32, 9, 9, 64, 45007)])
def test_long_rows_equal_their_pieces(dtype, H, Hkv, d, N):
    """Rows do not depend on one another: one call over many positions (hundreds of MB: other shares of a warp)
    and calls over a few hundred each write the same bits, forward and dx."""
    need_gpu()
    q, k, cos, sin, w, pos, gq, gk = _case(dtype, 1, N, H, Hkv, d, True, False, True, True, F32, seed=31, rows=4000)
    qo, ko = fa.qk_norm_rope(q, k, cos, sin, w[0], w[1], pos)
    dq, dk, _, _ = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos)
    for lo in list(range(0, N, 7919)) + [N - 301]:
        at = slice(lo, lo + 301)
        a, b = fa.qk_norm_rope(q[:, at], k[:, at], cos, sin, w[0], w[1], pos[:, at].contiguous())
        assert torch.equal(a, qo[:, at]) and torch.equal(b, ko[:, at])
        a, b, _, _ = fa.qk_norm_rope_bwd(q[:, at], k[:, at], cos, sin, gq[:, at], gk[:, at], w[0], w[1],
                                         pos[:, at].contiguous())
        assert torch.equal(a, dq[:, at]) and torch.equal(b, dk[:, at])
    assert fa.last_device_status()[0] == 0


def _dw_terms(x, cos, sin, pos, g, inter):
    """gr x r of every row [B, N, heads, d] in float64, on the tensors' device (zeros where padding is)."""
    x, g, d = x.double(), g.double(), x.shape[-1]
    at = torch.arange(x.shape[1], device=x.device).expand(x.shape[:2]) if pos is None else pos.long()
    c, s = (t.double()[at.clamp(min=0)][:, :, None] for t in (cos, sin))
    a, b = (slice(0, d, 2), slice(1, d, 2)) if inter else (slice(0, d // 2), slice(d // 2, d))
    gr = torch.empty_like(g)
    gr[..., a], gr[..., b] = g[..., a] * c + g[..., b] * s, g[..., b] * c - g[..., a] * s
    r = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    return torch.where((at >= 0)[:, :, None, None], gr * x * r, 0.0)


def _sums(x, cos, sin, pos, g, inter):
    """Sum and sum of magnitudes of the terms, a stretch of positions at a time."""
    out = torch.zeros((2, x.shape[-1]), dtype=torch.float64, device=x.device)
    for n in range(0, x.shape[1], 2048):
        at = slice(n, n + 2048)
        p = torch.arange(x.shape[1], device=x.device).expand(x.shape[:2]) if pos is None else pos
        t = _dw_terms(x[:, at], cos, sin, p[:, at], g[:, at], inter)
        out += torch.stack((t.sum((0, 1, 2)), t.abs().sum((0, 1, 2))))
    return out


def _depth(q, k):
    """How many fp32 additions a term of a gain's gradient goes through, at most.  The rows of q and k go in
    groups of 512 / d heads to 1776 resident warps (fewer where a warp would have less than two groups), by the
    groups of a position and one more: at least half of the share that the groups alone would give.  A lane adds its
    warp's groups one by one (a round of 4 and a rest more or less), then come the lanes of a feature (3), the
    warps of a block (4), and 64 bits."""
    n = 512 // q.shape[-1]
    groups = q.shape[0] * q.shape[1] * ((q.shape[2] + n - 1) // n + (k.shape[2] + n - 1) // n)
    return 2 * groups / 1776 + 5 + 3 + 4


LONG = [(BF, 2, 37, 5, 3, 128, True), (BF, 2, 3001, 8, 4, 64, False), (BF, 1, 3301, 33, 5, 128, False),
        (F32, 1, 3301, 33, 5, 128, True), (BF, 1, 20001, 33, 7, 128, False), (BF, 1, 40009, 4, 1, 64, True),
        (F32, 1, 45007, 9, 9, 64, False), (BF, 4, 1001, 16, 4, 64, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("one_sign", [True, False])
@pytest.mark.parametrize("dtype,B,N,H,Hkv,d,inter", LONG)
def test_gain_gradients_to_the_depth_of_their_sums(dtype, B, N, H, Hkv, d, inter, one_sign):
    """dw against a float64 sum, with 2^-24 for every fp32 addition that a term goes through (``_depth``), 32 for what
    went into the term (the module's docstring counts fewer), and the last rounding.  With gradients
    along the rotated rows all terms have one sign, so that a group of rows left out, or counted
    twice, anywhere, is further off than that (in the calls over more than 10000 positions the groups of 16)."""
    need_gpu()
    q, k, cos, sin, w, pos, gq, gk = _case(dtype, B, N, H, Hkv, d, True, inter, True, True, F32, seed=26)
    if one_sign:
        gq, gk = fa.qk_norm_rope_fwd(q, k, cos, sin, positions=pos, interleaved=inter)
    got = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos, interleaved=inter)[2:]
    for x, g, dw in ((q, gq, got[0]), (k, gk, got[1])):
        ref, mag = _sums(x, cos, sin, pos, g, inter)
        tol = 2.0 ** -24 * ((_depth(q, k) + 32) * mag + ref.abs())
        assert bool(((dw.double() - ref).abs() <= tol).all())
        if one_sign:  # what one group of rows adds shows in some feature
            m = 16 if N > 10000 else 1
            at = torch.nonzero(pos[0] >= 0)[:, 0]
            at = at[:at.numel() // m * m].view(-1, m)[:: max(1, N // (200 * m))].flatten()
            t = _dw_terms(x[:1, at], cos, sin, pos[:1, at], g[:1, at], inter)[0]
            last = t[:, (x.shape[2] - 1) // (512 // d) * (512 // d):].sum(1)  # the last group, not always full
            assert bool((last.view(-1, m, d).sum(1).abs() > 2 * tol).any(-1).all())
    if N == 37:  # the float64 sums themselves
        for x, g in ((q, gq), (k, gk)):
            ref = torch.from_numpy(S.norm_rope_backward(_f(x), np.ones(d), _f(cos), _f(sin), _f(g), pos.cpu().numpy(), 1e-6, inter)[1])
            assert torch.allclose(_sums(x, cos, sin, pos, g, inter)[0].cpu(), ref, rtol=1e-12, atol=1e-12)


@pytest.mark.gpu
def test_gain_gradients_of_rows_beyond_32_bit_offsets():
    """Rows at the start, across element 2^31 and at the end of 2.3e9; the others are zeros, which add exactly
    nothing: their sums in float64."""
    need_gpu()
    N, H, d, n = 280000, 64, 128, 37
    g = torch.Generator().manual_seed(27)
    q = torch.zeros((1, N, H, d), dtype=BF, device="cuda")
    k = torch.zeros((1, N, 1, d), dtype=BF, device="cuda")
    cos, sin = fa.rope_tables(N, d)
    w = (1 + 0.3 * torch.randn(d, generator=g)).cuda()
    middle = 2 ** 31 // (H * d) - n // 2
    rows = torch.cat([torch.arange(a, a + n) for a in (0, middle, N - n)]).cuda()
    q[:, rows] = torch.randn((1, 3 * n, H, d), generator=g).to(BF).cuda()
    k[:, rows] = torch.randn((1, 3 * n, 1, d), generator=g).to(BF).cuda()
    gq, gk = fa.qk_norm_rope_fwd(q, k, cos, sin)
    got = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w, w)[2:]
    for x, y, dw in ((q, gq, got[0]), (k, gk, got[1])):
        ref, mag = _sums(x[:, rows], cos, sin, rows.view(1, -1), y[:, rows], False)
        assert bool(((dw.double() - ref).abs() <= 2.0 ** -24 * ((3 * n * 16 + 39) * mag + ref.abs())).all())


@pytest.mark.gpu
def test_gain_gradients_where_one_output_is_used():
    """Only k's output in the loss: its gain's gradient is the sum over k's rows, q's gain gets zeros."""
    need_gpu()
    q, k, cos, sin, w, pos, _, gk = _case(F32, 2, 9, 3, 2, 64, True, False, False, True, F32, seed=28)
    k, wq, wk = (t.clone().requires_grad_(True) for t in (k, *w))
    _, ko = fa.qk_norm_rope(q, k, cos, sin, wq, wk, pos)
    dk, dwq, dwk = torch.autograd.grad(ko, (k, wq, wk), gk)
    _check_bwd(k, wk, cos, sin, pos, False, gk, dk, dwk)
    ref, mag = _sums(k.detach(), cos, sin, pos, gk, False)
    assert bool(((dwk.double() - ref).abs() <= 2.0 ** -24 * ((_depth(q, k) + 32) * mag + ref.abs())).all())
    assert torch.count_nonzero(dwq) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences_of_the_kernel(inter):
    """Central differences of the fp32 forward itself.  Step 2^-7: the forward's error, 2^-20 of
    values around 4, over the step gives 2^-11 per element of a sum of 16 outputs; the third
    derivative of a normalised row times h^2 / 6 stays under 2^-13."""
    need_gpu()
    q, k, cos, sin, w, pos, gq, gk = _case(F32, 1, 2, 1, 1, 64, True, inter, False, False, F32, seed=14)
    dq, _, dwq, _ = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], interleaved=inter)

    def loss(q, wq):
        out = fa.qk_norm_rope_fwd(q, k, cos, sin, wq, w[1], interleaved=inter)[0]
        return float((out.double() * gq.double()).sum())

    h = 2.0 ** -7
    for i in (0, 3, 31, 32, 63):
        e = torch.zeros_like(q)
        e[0, 1, 0, i] = h
        assert abs((loss(q + e, w[0]) - loss(q - e, w[0])) / (2 * h) - float(dq[0, 1, 0, i])) <= 2.0 ** -7
        e = torch.zeros_like(w[0])
        e[i] = h
        assert abs((loss(q, w[0] + e) - loss(q, w[0] - e)) / (2 * h) - float(dwq[i])) <= 2.0 ** -7


@pytest.mark.gpu
def test_autograd_of_the_whole_step_before_attention():
    """A packed projection, norm and rotation, then causal attention with shared K/V heads: the
    gradients that autograd returns.  The attention's are held to its own bar, max |d| / max |ref| <= 2e-2,
    on the q, k that it was given; the norm's projection can at most double a relative error of
    the largest element, and the sum over rows does not raise it: 4e-2."""
    need_gpu()
    B, N, H, Hkv, d = 2, 200, 4, 2, 128
    g = torch.Generator().manual_seed(15)
    x = torch.randn((B, N, H + 2 * Hkv, d), generator=g).to(BF).cuda().requires_grad_(True)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).cuda().requires_grad_(True) for _ in range(2))
    cos, sin = fa.rope_tables(N, d)
    do = torch.randn((B, N, H, d), generator=g).to(BF).cuda()
    q, k, v = x.split((H, Hkv, Hkv), dim=2)
    qr, kr = fa.qk_norm_rope(q, k, cos, sin, wq, wk)
    o = fa.attention(qr, kr, v.contiguous(), causal=True)
    o.backward(do)
    scale = float(np.float32(1 / np.sqrt(d)))
    rq, rk, rv = oracle.backward(_f(qr), _f(kr), _f(v), _f(do), scale, True)
    dxq, dwq = S.norm_rope_backward(_f(q), _f(wq), _f(cos), _f(sin), rq)
    dxk, dwk = S.norm_rope_backward(_f(k), _f(wk), _f(cos), _f(sin), rk)
    got = _f(x.grad)
    for a, ref in ((got[:, :, :H], dxq), (got[:, :, H:H + Hkv], dxk), (got[:, :, H + Hkv:], rv), (_f(wq.grad), dwq),
                   (_f(wk.grad), dwk)):
        assert np.max(np.abs(a - ref)) <= 4e-2 * np.max(np.abs(ref))


@pytest.mark.gpu
def test_autograd_of_broadcast_and_missing_gradients():
    need_gpu()
    q, k, cos, sin, w, pos, _, _ = _case(BF, 2, 9, 3, 2, 64, True, False, False, True, BF, seed=16)
    leaves = [t.requires_grad_(True) for t in (q, k, *w)]
    qo, ko = fa.qk_norm_rope(q, k, cos, sin, w[0], w[1], pos)
    qo.sum().backward()                       # an expanded gradient for q, none for k
    one = torch.ones_like(q)
    _check_bwd(q, w[0], cos, sin, pos, False, one, q.grad, w[0].grad)
    assert torch.count_nonzero(k.grad) == 0 and torch.count_nonzero(w[1].grad) == 0
    # a gradient that the kernels cannot read in place: an odd offset, then transposed features
    for g in (torch.randn(q.numel() + 1, device="cuda").to(BF)[1:].view(q.shape),
              torch.randn((*q.shape[:2], q.shape[3], q.shape[2]), device="cuda").to(BF).transpose(2, 3)):
        qo, _ = fa.qk_norm_rope(q, k, cos, sin, w[0], w[1], pos)
        dq, dw = torch.autograd.grad(qo, (q, w[0]), g)
        _check_bwd(q, w[0], cos, sin, pos, False, g, dq, dw)
    # one leaf alone
    k2 = k.detach().requires_grad_(True)
    _, ko = fa.qk_norm_rope(q.detach(), k2, cos, sin, w[0].detach(), w[1].detach(), pos)
    dk, = torch.autograd.grad(ko, k2, torch.ones_like(ko))
    _check_bwd(k, w[1], cos, sin, pos, False, torch.ones_like(k), dk, w[1].grad * 0 + dk.new_tensor(_dw(k, w[1], cos, sin, pos)))
    with pytest.raises(RuntimeError):         # no second derivative
        qo, _ = fa.qk_norm_rope(*leaves[:2], cos, sin, *leaves[2:], pos)
        gq, = torch.autograd.grad(qo.float().square().sum(), leaves[0], create_graph=True)
        gq.sum().backward()


def _dw(x, w, cos, sin, pos):
    return S.norm_rope_backward(_f(x), _f(w), _f(cos), _f(sin), np.ones_like(_f(x)), pos.cpu().numpy())[1]


@pytest.mark.gpu
def test_padding_is_neither_read_nor_left_behind():
    need_gpu()
    q, k, cos, sin, w, _, gq, gk = _case(BF, 2, 12, 4, 2, 128, True, False, False, False, BF, seed=17)
    pos = torch.arange(12, dtype=torch.int32).repeat(2, 1)
    pos[0, 5:] = -1
    pos[1, :3] = -7
    pad = (pos < 0).cuda()
    pos = pos.cuda()
    for t in (q, k, gq, gk):
        t[pad] = float("nan")
    out = [torch.full_like(t, float("nan")) for t in (q, k)]
    qo, ko = fa.qk_norm_rope_fwd(q, k, cos, sin, w[0], w[1], pos, q_out=out[0], k_out=out[1])
    grads = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos)
    for t in (qo, ko, *grads):
        assert torch.isfinite(t).all()
    for t in (qo, ko, grads[0], grads[1]):
        assert torch.count_nonzero(t[pad]) == 0


@pytest.mark.gpu
def test_far_positions_are_reported_and_treated_as_padding():
    need_gpu()
    q, k, cos, sin, w, _, gq, gk = _case(BF, 1, 6, 4, 2, 64, True, False, False, False, BF, seed=18)
    pos = torch.tensor([[0, 1, cos.shape[0], 3, 2 ** 31 - 1, 5]], dtype=torch.int32).cuda()
    fa.last_device_status()
    qo, _ = fa.qk_norm_rope(q, k, cos, sin, w[0], w[1], pos)
    rc, detail = fa.last_device_status()
    assert rc == -9 and detail == 0x2000 | 0xD3
    good = pos.clone()
    good[pos >= cos.shape[0]] = -1
    assert torch.equal(qo, fa.qk_norm_rope(q, k, cos, sin, w[0], w[1], good)[0])
    dq = fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos)[0]
    assert fa.last_device_status()[0] == -9
    assert torch.count_nonzero(dq[0, [2, 4]]) == 0 and torch.isfinite(dq).all()
    assert fa.last_device_status()[0] == 0


@pytest.mark.gpu
def test_empty_problems():
    need_gpu()
    cos, sin = fa.rope_tables(4, 64)
    w = torch.ones(64, device="cuda")
    for B, N, H, Hkv in ((0, 3, 2, 1), (2, 0, 2, 1), (2, 3, 0, 0)):
        q, k = torch.empty((B, N, H, 64), device="cuda"), torch.empty((B, N, Hkv, 64), device="cuda")
        qo, ko = fa.qk_norm_rope(q, k, cos, sin, w, w)
        assert qo.shape == q.shape and ko.shape == k.shape
        dq, dk, dwq, dwk = fa.qk_norm_rope_bwd(q, k, cos, sin, q, k, w, w)
        assert torch.count_nonzero(dwq) == 0 and torch.count_nonzero(dwk) == 0
        assert fa.qk_norm_rope_bwd(q, k, cos, sin, q, k)[2] is None


@pytest.mark.gpu
def test_strides_that_the_kernels_cannot_read_are_refused():
    need_gpu()
    q, k, cos, sin, w, _, gq, gk = _case(BF, 2, 3, 4, 2, 64, True, False, False, False, BF, seed=22)
    wide = torch.zeros(2, 3, 4, 128, dtype=BF, device="cuda")[..., ::2]
    with pytest.raises(ValueError, match="contiguous"):
        fa.qk_norm_rope(wide, k, cos, sin)
    odd = torch.zeros(2, 3, 4, 68, dtype=BF, device="cuda")[..., :64]
    with pytest.raises(ValueError, match="16 bytes"):
        fa.qk_norm_rope(odd, k, cos, sin)
    with pytest.raises(ValueError, match="16 bytes"):
        fa.qk_norm_rope_bwd(q, k, cos, sin, odd, gk)
    with pytest.raises(fa.FAError) as e:                   # base not 16-byte aligned
        fa.qk_norm_rope(torch.zeros(q.numel() + 1, dtype=BF, device="cuda")[1:].view(q.shape), k, cos, sin)
    assert e.value.status == -3
    with pytest.raises(ValueError, match="q_out"):
        fa.qk_norm_rope_fwd(q, k, cos, sin, q_out=q.float())
    # what they can: heads and positions in another order, one row for all (stride 0)
    t = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert not t.is_contiguous() and torch.equal(fa.qk_norm_rope(t, k, cos, sin, *w)[0], fa.qk_norm_rope(q, k, cos, sin, *w)[0])
    e = q[:, :, :1].expand(2, 3, 4, 64)
    assert torch.equal(fa.qk_norm_rope(e, k, cos, sin, *w)[0], fa.qk_norm_rope(e.contiguous(), k, cos, sin, *w)[0])


@pytest.mark.gpu
def test_nan_and_inf_stay_in_their_rows():
    need_gpu()
    q, k, cos, sin, w, _, _, _ = _case(BF, 1, 4, 8, 2, 128, True, False, False, False, BF, seed=19)
    clean = fa.qk_norm_rope(q, k, cos, sin, w[0], w[1])[0]
    q = q.clone()
    q[0, 1, 2, 5] = float("nan")
    q[0, 2, 7, 100] = float("inf")
    out = fa.qk_norm_rope(q, k, cos, sin, w[0], w[1])[0]
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, 1, 2], hit[0, 2, 7] = True, True
    assert torch.isnan(out[0, 1, 2]).all() and torch.isnan(out[0, 2, 7]).any()
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("N", [3, 2000])
@pytest.mark.parametrize("captured", [False, True])
def test_tables_rewritten_right_before_the_call(N, captured):
    """The kernels come up while the one before ends: each call reads the tables, gains and rows as that one left
    them, also where the call before it had read the old ones."""
    need_gpu()
    q, k, cos, sin, w, pos, gq, gk = _case(BF, 1, N, 8, 2, 128, True, False, False, False, F32, seed=25)
    cos0, sin0, q0 = cos.clone(), sin.clone(), q.clone()
    steps = []
    for _ in range(4):
        cos0, sin0, q0 = -sin0, cos0, q0 * -0.5
        steps.append((cos0, sin0, q0, fa.qk_norm_rope_fwd(q0, k, cos0, sin0, w[0], w[1]),
                      fa.qk_norm_rope_bwd(q0, k, cos0, sin0, gq, gk, w[0], w[1])))

    def run():
        out = []
        for c, s, x, _, _ in steps:
            cos.copy_(c), sin.copy_(s), q.copy_(x)
            out.append(fa.qk_norm_rope_fwd(q, k, cos, sin, w[0], w[1]))
            cos.copy_(c), sin.copy_(s)
            out.append(fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1]))
        return out

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        for _ in range(20):
            graph.replay()
    else:
        for _ in range(20):
            out = run()
    for (_, _, _, fwd, bwd), a, b in zip(steps, out[0::2], out[1::2]):
        assert all(torch.equal(x, y) for x, y in zip((*fwd, *bwd), (*a, *b)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,inter,d", [(BF, False, 128), (F32, True, 64)])
def test_autograd_of_the_rotation_alone(dtype, inter, d):
    need_gpu()
    q, k, cos, sin, w, pos, gq, gk = _case(dtype, 2, 21, 5, 2, d, False, inter, True, False, F32, seed=29)
    q, k = q.detach().requires_grad_(True), k.detach().requires_grad_(True)
    qo, ko = fa.qk_norm_rope(q, k, cos, sin, interleaved=inter)
    dq, dk = torch.autograd.grad((qo, ko), (q, k), (gq, gk))
    _check_bwd(q, None, cos, sin, pos, inter, gq, dq, None)
    _check_bwd(k, None, cos, sin, pos, inter, gk, dk, None)
    with pytest.raises(RuntimeError):         # no second derivative here either
        qo, _ = fa.qk_norm_rope(q, k, cos, sin, interleaved=inter)
        dq, = torch.autograd.grad(qo.float().square().sum(), q, create_graph=True)
        dq.sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,H,Hkv", [(0, 3, 2, 1), (2, 0, 2, 1), (2, 3, 0, 0), (2, 3, 0, 2)])
@pytest.mark.parametrize("norm", [True, False])
def test_autograd_of_empty_tensors(B, N, H, Hkv, norm):
    need_gpu()
    cos, sin = fa.rope_tables(4, 64)
    leaves = [torch.ones((B, N, h, 64), device="cuda", requires_grad=True) for h in (H, Hkv)]
    if norm:
        leaves += [torch.ones(64, device="cuda", requires_grad=True) for _ in range(2)]
    qo, ko = fa.qk_norm_rope(leaves[0], leaves[1], cos, sin, *leaves[2:])
    (qo.sum() + ko.sum()).backward()
    for t in leaves:
        assert t.grad.shape == t.shape and torch.isfinite(t.grad).all()
    if norm:
        assert torch.count_nonzero(leaves[2].grad) == 0
        assert (torch.count_nonzero(leaves[3].grad) > 0) == (B * N * Hkv > 0)


@pytest.mark.gpu
def test_a_training_step_captured():
    """Forward and backward through autograd in one graph, replayed on new rows and gradients."""
    need_gpu()
    q, k, cos, sin, w, pos, gq, gk = _case(BF, 2, 40, 6, 2, 128, True, False, False, True, F32, seed=30)
    new = _case(BF, 2, 40, 6, 2, 128, True, False, False, True, F32, seed=31)
    want = [fa.qk_norm_rope_bwd(a, b, cos, sin, c, e, w[0], w[1], pos) for a, b, c, e in
            ((q, k, gq, gk), (new[0], new[1], new[6], new[7]))]
    leaves = [t.clone().requires_grad_(True) for t in (q, k, *w)]

    def step():
        qo, ko = fa.qk_norm_rope(leaves[0], leaves[1], cos, sin, leaves[2], leaves[3], pos)
        return torch.autograd.grad((qo, ko), leaves, (gq, gk))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want[0]))
    with torch.no_grad():
        for t, u in ((leaves[0], new[0]), (leaves[1], new[1]), (gq, new[6]), (gk, new[7])):
            t.copy_(u)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want[1]))


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    """One graph of forward and backward, replayed on new inputs; and the calls on a side stream."""
    need_gpu()
    q, k, cos, sin, w, pos, gq, gk = _case(BF, 2, 40, 6, 2, 128, True, False, False, True, BF, seed=20)
    q2, k2, _, _, _, _, gq2, gk2 = _case(BF, 2, 40, 6, 2, 128, True, False, False, True, BF, seed=21)

    def both():
        return (*fa.qk_norm_rope_fwd(q, k, cos, sin, w[0], w[1], pos),
                *fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos))

    want = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*fa.qk_norm_rope_fwd(q, k, cos, sin, w[0], w[1], pos, stream=side),
           *fa.qk_norm_rope_bwd(q, k, cos, sin, gq, gk, w[0], w[1], pos, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    graph.replay()
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    for t, u in ((q, q2), (k, k2), (gq, gq2), (gk, gk2)):
        t.copy_(u)
    graph.replay()
    for a, b in zip(out, both()):
        assert torch.equal(a, b)
