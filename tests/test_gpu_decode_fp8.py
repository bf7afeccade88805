"""Decode over the paged 8-bit cache: the CUDA kernels against the fp64 oracle on the dequantised rows.

Tolerance of an output element: half a bf16 step, 2^-8 of it; and, against sum_j p_j |v_j|
(the oracle run on |V|): the f16 rounding of P times the V scale, 2^-11; the
fp32 sums and ex2 (2 units), under 2^-16; and e^delta - 1 for an error delta of the scores, which
moves a probability and the denominator, so 2 delta.  delta: fp32 accumulation of d = 128 products
on the tensor cores, 2^-23 of the magnitudes each: 2^-16 scale sum |q k|, with ex2's own argument rounding
(2^-24 of the score) far below.  Doubled once for the second-order terms.
LSE: delta + 2^-18 (1 + |LSE|) + the fp32 sum of the row's p, 2^-24 for each of L / 32 + 64 steps.
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import exact_io_aware_51_b200 as fa
from exact_io_aware_51_b200 import inputs as I
from oracle import serving as S
from tests.helpers import need_gpu


def _make(B, H, Hkv, d, P, lens, seed, spare=2, max_pages=None, spread=1.0, poison=True):
    """q, codes, scales, table, lens on the CPU; unused rows hold NaN codes and NaN scales."""
    q, k, v, table, sl = I.make_paged_decode(B, H, Hkv, d, P, lens, seed=seed, spare_pages=spare, max_pages=max_pages)
    g = torch.Generator().manual_seed(seed + 1)
    k, v = (t.float() * torch.exp(spread * torch.randn((*t.shape[:3], 1), generator=g)) for t in (k, v))
    kc, kb = S.quantise_rows(k.to(torch.bfloat16).double().numpy())
    vc, vb = S.quantise_rows(v.to(torch.bfloat16).double().numpy())
    if poison:
        used = np.zeros(k.shape[:2], bool)
        for b, n in enumerate(lens):
            for j in range(n):
                used[int(table[b, j // P]), j % P] = True
        for c, s in ((kc, kb), (vc, vb)):
            c[~used], s[~used] = 0xFF, 255
    sc = np.stack([np.moveaxis(kb, 1, 2), np.moveaxis(vb, 1, 2)], axis=2)
    return q, torch.from_numpy(kc), torch.from_numpy(vc), torch.from_numpy(np.ascontiguousarray(sc)), table, sl


def _check(args, o, lse, scale, window=None, skip=()):
    q, kc, vc, sc, table, sl = args
    K, V = S.dequantise_cache(kc, vc, sc)
    ro, rl = S.decode_window(q.double(), K, V, table, sl, scale, window)
    mo, _ = S.decode_window(q.double(), K, np.abs(V), table, sl, scale, window)
    P = kc.shape[1]
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    for b, n in enumerate(int(x) for x in sl):
        if b in skip:
            continue
        if n == 0:
            assert np.all(o[b] == 0) and np.all(np.isneginf(lse[b]))
            continue
        lo = 0 if window is None else max(0, n - 1 - window)
        at = np.arange(lo, n)
        k = np.abs(K[table[b, at // P].numpy(), at % P])                       # [n, Hkv, d]
        a = np.abs(q[b].double().numpy()).reshape(k.shape[1], -1, k.shape[2])  # [Hkv, G, d]
        delta = 2.0 ** -16 * scale * np.einsum("hgd,nhd->hgn", a, k).max(-1).reshape(-1)
        tol = 2.0 ** -8 * np.abs(ro[b]) + 2 * (2.0 ** -11 + 2.0 ** -16 + 2 * delta[:, None]) * mo[b] + 1e-30
        assert np.all(np.abs(o[b] - ro[b]) <= tol), b
        assert np.all(np.abs(lse[b] - rl[b]) <= delta + 2.0 ** -18 * (1 + np.abs(rl[b])) + 2.0 ** -24 * (n / 32 + 64)), b


def _run(args, **kw):
    q, kc, vc, sc, table, sl = (t.cuda() for t in args)
    o, lse = fa.decode_paged_fp8(q, kc, vc, sc, table, sl, **kw)
    assert fa.last_device_status()[0] == 0
    return o, lse


CASES = [
    # B, H, Hkv, d, page, lengths, window
    (4, 8, 2, 128, 16, [1, 17, 64, 200], None),
    (3, 16, 16, 64, 8, [0, 65, 130], None),
    (2, 32, 1, 128, 64, [300, 129], None),          # 32 query heads on one K/V head: two head groups
    (2, 64, 8, 128, 256, [1000, 513], None),
    (2, 32, 2, 64, 32, [63, 777], None),            # 16 query heads per K/V head: two column blocks
    (1, 4, 4, 64, 4096, [5000], None),
    (5, 12, 4, 128, 128, [128, 129, 0, 255, 1], None),
    (2, 9, 1, 128, 16, [127, 257], None),           # 9: the second column block holds one head
    (2, 20, 1, 64, 16, [40, 383], None),            # 20: two groups, the second with 4
    (3, 8, 2, 128, 16, [500, 130, 3], 0),
    (3, 8, 2, 64, 8, [500, 130, 0], 127),
    (2, 16, 2, 128, 16, [900, 385], 256),
    (2, 5, 5, 128, 512, [1500, 100], 1000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=[f"B{c[0]}H{c[1]}kv{c[2]}d{c[3]}P{c[4]}w{c[6]}" for c in CASES])
def test_decode_matches_oracle(case):
    need_gpu()
    B, H, Hkv, d, P, lens, window = case
    args = _make(B, H, Hkv, d, P, lens, seed=sum(lens) % 97)
    scale = float(np.float32(1 / math.sqrt(d)))
    o, lse = _run(args, scale=scale, window_left=window)
    _check(args, o, lse, scale, window)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [None, 6000])
def test_split_and_unsplit(d, window):
    """Long sequences in a small batch, with and without a workspace, and with one that holds fewer chunks."""
    need_gpu()
    lens = [9000, 3, 4100]
    B, H, Hkv, P = 3, 8, 2, 16
    args = _make(B, H, Hkv, d, P, lens, seed=4)
    size = fa.decode_fp8_workspace_size(B, H, Hkv, d, P, args[4].shape[1], window)
    assert size > 0
    for n in (None, 16, size // 2):
        ws = None if n is None else torch.empty(n, dtype=torch.uint8, device="cuda")
        o, lse = _run(args, scale=0.1, window_left=window, workspace=ws)
        _check(args, o, lse, 0.1, window)


@pytest.mark.gpu
def test_same_bits_twice():
    need_gpu()
    args = _make(4, 16, 4, 128, 16, [700, 64, 1, 5000], seed=8)
    a, b = _run(args), _run(args)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("H", [8, 16])
def test_growing_scores_and_scales(H):
    """Scores that grow along the positions (the reference has to move) and V rows whose scales span
    2^-40 to 2^40, growing and shrinking; queries from 2^-60 to 2^30."""
    need_gpu()
    d, P, lens = 128, 16, [1500, 700]
    q, k, v, table, sl = I.make_paged_decode(2, H, 1, d, P, lens, seed=9)
    k, v = k.double().numpy(), v.double().numpy()
    for b, n in enumerate(lens):
        for j in range(n):
            pg, s = int(table[b, j // P]), j % P
            k[pg, s] *= (j + 1) / n * 4
            v[pg, s] *= 2.0 ** (40 * math.sin(j / 90.0 + b))
    kc, kb = S.quantise_rows(k)
    vc, vb = S.quantise_rows(v)
    sc = np.ascontiguousarray(np.stack([np.moveaxis(kb, 1, 2), np.moveaxis(vb, 1, 2)], axis=2))
    args = (q, torch.from_numpy(kc), torch.from_numpy(vc), torch.from_numpy(sc), table, sl)
    o, lse = _run(args, scale=0.3)
    _check(args, o, lse, 0.3)
    for e in (-60, 30):
        args = (q * 2.0 ** e, *args[1:])
        scale = 0.3 * 2.0 ** -e
        o, lse = _run(args, scale=scale)
        _check(args, o, lse, scale)
        args = (q, *args[1:])


def _planted(x, v, H, d, P, seed):
    """Decode arguments of one sequence whose head scores are the rows x [n] (on the e4m3 grid times a power of
    two) and whose V rows are v [n, d]: q is the first unit vector, K holds x in that feature."""
    n = len(x)
    g = torch.Generator().manual_seed(seed)
    pages = (n + P - 1) // P
    table = torch.randperm(pages, generator=g).to(torch.int32).view(1, pages)
    k, w = np.zeros((pages, P, 1, d)), np.zeros((pages, P, 1, d))
    for j in range(n):
        k[int(table[0, j // P]), j % P, 0, 0] = x[j]
        w[int(table[0, j // P]), j % P, 0] = v[j]
    kc, kb = S.quantise_rows(k)
    vc, vb = S.quantise_rows(w)
    sc = np.ascontiguousarray(np.stack([np.moveaxis(kb, 1, 2), np.moveaxis(vb, 1, 2)], axis=2))
    q = torch.zeros((1, H, d), dtype=torch.bfloat16)
    q[:, :, 0] = 1
    return q, torch.from_numpy(kc), torch.from_numpy(vc), torch.from_numpy(sc), table, torch.tensor([n], dtype=torch.int32)


def _unlike_rows(n, d, what, seed):
    """Scores (natural logarithms of the probabilities but for a constant) and V rows in which few rows are of
    a size far from the others'."""
    rng = np.random.default_rng(seed)
    x, v = rng.integers(0, 2, n) * -1.0, rng.standard_normal((n, d))
    if what.startswith("unlikely"):       # one large row that its probability makes small again, or nothing
        bits, nats = {"unlikely28": (28, 22.0), "unlikely40": (40, 40.0), "unlikely100": (100, 72.0)}[what]
        v[n // 3] *= 2.0 ** bits
        x[n // 3] = -nats
    elif what == "sparse":                # a likely large row that is zero in most features
        v[n // 3] *= 2.0 ** 34
        v[n // 3, 5:] = 0
    elif what == "later":                 # the second half larger by what its probability is smaller
        v[n // 2:] *= 2.0 ** 30
        x[n // 2:] -= 20.0
    elif what == "earlier":
        v[:n // 2] *= 2.0 ** 30
        x[:n // 2] -= 20.0
    elif what == "sink":                  # nearly all probability on a row of zeros
        v[0] = 0
        x[1:] -= 24.0
    else:
        assert what == "huge and small"
        v *= 2.0 ** -60
        v[n // 3, :3] = 2.0 ** 100
        v[n // 3, 3:] = 0
    return x, v


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["unlikely28", "unlikely40", "unlikely100", "sparse", "later", "earlier", "sink",
                                  "huge and small"])
@pytest.mark.parametrize("n,H,d", [(20, 4, 128), (700, 8, 64), (700, 16, 128), (300, 12, 64), (5000, 8, 128)])
def test_v_rows_of_very_different_size(what, n, H, d):
    """The bound of every other case holds where few V rows are of a size far from the others': unlikely and large,
    large in few features, zeros that take the probability; in one tile, in several, and in several ranges."""
    need_gpu()
    args = _planted(*_unlike_rows(n, d, what, seed=n), H, d, 16, seed=17)
    for window in (None, n - 2):
        o, lse = _run(args, scale=1.0, window_left=window)
        _check(args, o, lse, 1.0, window)


@pytest.mark.gpu
@pytest.mark.parametrize("d,H", [(128, 8), (64, 32)])
def test_small_queries_on_large_keys_and_the_reverse(d, H):
    """Scores of ordinary size whose factors are up to 2^115 away from it."""
    need_gpu()
    args = _make(2, H, 2, d, 16, [300, 129], seed=18, poison=False)
    q, kc, vc, sc, table, sl = args
    q = torch.where(q.abs() < 2.0 ** -4, torch.tensor(2.0 ** -4, dtype=q.dtype), q)  # no subnormals below
    want = _run((q, *args[1:]), scale=0.2)
    for e in (115, 60, -60, -110):
        s2 = sc.clone()
        s2[:, :, 0] = (sc[:, :, 0].int() + e).to(torch.uint8)
        got = (q * 2.0 ** -e, kc, vc, s2, table, sl)
        assert torch.equal(got[0].double(), q.double() * 2.0 ** -e)
        o, lse = _run(got, scale=0.2)
        _check(got, o, lse, 0.2)
        if e > -110:  # only powers of two have moved (at -110 the smallest scores are subnormal on the way)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("n,H,d", [(6, 8, 128), (6, 32, 64), (900, 8, 64)])
@pytest.mark.parametrize("e", [24, 40, 118])
def test_scores_so_large_that_one_row_takes_all(n, H, d, e):
    """Scores of 2^e, far apart: the output is the V row of the largest.  LSE is that score, scale log2(e) rounded
    once, its product with the score, and ln 2 times that, once each: 4 * 2^-24 of it."""
    need_gpu()
    rng = np.random.default_rng(n)
    x = rng.choice([1.0, 1.25, -3.5, 2.0, 0.0], n) * 2.0 ** e
    x[n - 4] = 3.0 * 2.0 ** e
    args = _planted(x, rng.standard_normal((n, d)), H, d, 16, seed=19)
    o, lse = _run(args, scale=0.25)
    V = S.dequantise_cache(*args[1:4])[1]
    want = torch.from_numpy(V[int(args[4][0, (n - 4) // 16]), (n - 4) % 16, 0]).to(torch.bfloat16)
    for h in range(H):
        assert torch.equal(o.cpu()[0, h], want)
        assert abs(float(lse[0, h]) - 0.75 * 2.0 ** e) <= 2.0 ** -22 * 0.75 * 2.0 ** e


@pytest.mark.gpu
def test_nan_rows_reach_the_heads_that_see_them():
    need_gpu()
    args = _make(2, 8, 2, 128, 16, [300, 300], seed=10)
    q, kc, vc, sc, table, sl = args
    clean = _run(args)
    for which in (0, 1):
        s2 = sc.clone()
        s2[int(table[1, 5]), 1, which, 7] = 255       # position 87 of sequence 1, K/V head 1
        o, lse = _run((q, kc, vc, s2, table, sl))
        assert torch.isnan(o[1, 4:].float()).all()
        assert torch.equal(o[0], clean[0][0]) and torch.equal(o[1, :4], clean[0][1, :4])
        if which == 0:
            assert torch.isnan(lse[1, 4:]).all()
        # behind the sequence's end, or before its window, it is not seen
        short = sl.clone()
        short[1] = 87
        o, lse = _run((q, kc, vc, s2, table, short))
        assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
        o, _ = _run((q, kc, vc, s2, table, sl), window_left=300 - 1 - 88)
        assert torch.isfinite(o.float()).all()
    # a NaN code of K makes the heads NaN, one of V its feature; behind the end neither does
    for cache, hit in ((0, slice(None)), (1, slice(37, 38))):
        pools = [kc.clone(), vc.clone()]
        pools[cache][int(table[1, 5]), 7, 1, 37] = 0xFF
        o, _ = _run((q, *pools, sc, table, sl))
        assert torch.isnan(o[1, 4:, hit].float()).all()
        if cache == 1:
            rest = [f for f in range(128) if f != 37]
            assert torch.equal(o[1, 4:][:, rest], clean[0][1, 4:][:, rest])
        assert torch.equal(o[0], clean[0][0]) and torch.equal(o[1, :4], clean[0][1, :4])
        o, _ = _run((q, *pools, sc, table, short))
        assert torch.isfinite(o.float()).all()
    # a query of NaN, and one of Inf
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[0, 3, 9] = bad
        o, _ = _run((q2, kc, vc, sc, table, sl))
        assert torch.isnan(o[0, 3].float()).all()
        keep = torch.ones(2, 8, dtype=torch.bool)
        keep[0, 3] = False
        assert torch.equal(o.cpu()[keep], clean[0].cpu()[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("what", ["page_index", "negative_page", "length", "negative_length"])
def test_out_of_range_device_inputs(what, split):
    need_gpu()
    lens = [100, 5000, 80] if split else [100, 50, 80]
    B, H, Hkv, d, P = 3, 8, 2, 64, 16
    args = _make(B, H, Hkv, d, P, lens, seed=12)
    table, sl = args[4].clone(), args[5].clone()
    if what == "page_index":
        table[1, 2] = args[1].shape[0] + 5
    elif what == "negative_page":
        table[1, 0] = -1
    else:
        sl[1] = table.shape[1] * P + 1 if what == "length" else -3
    assert (fa.decode_fp8_workspace_size(B, H, Hkv, d, P, table.shape[1]) > 0) == split
    fa.last_device_status()
    o, lse = fa.decode_paged_fp8(*(t.cuda() for t in (*args[:4], table, sl)), scale=0.1)
    rc, detail = fa.last_device_status()
    assert rc == -9 and detail == 0x2000 | (0xD2 if "page" in what else 0xD1)
    assert torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1]))
    _check(args, o, lse, 0.1, skip=(1,))


@pytest.mark.gpu
def test_pages_before_the_window_are_not_looked_up():
    """A cache that gives back pages behind its window leaves anything in their table entries."""
    need_gpu()
    args = _make(2, 8, 2, 128, 16, [700, 300], seed=13)
    q, kc, vc, sc, table, sl = args
    whole = _run(args)
    for w in (699, 2 ** 20, 2 ** 40):                 # windows longer than every sequence
        got = _run(args, window_left=w)
        assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])
    want = _run(args, window_left=100)
    t = table.clone()
    for b, n in enumerate((700, 300)):
        t[b, :(n - 1 - 100) // 16] = 2 ** 30
    got = _run((q, kc, vc, sc, t, sl), window_left=100)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_full_size_sampled_sequences():
    """64 sequences of 512 to 8192 positions, 64 query heads on 8 K/V heads, pages handed out by cache_append's
    own quantisation: six sequences against the oracle."""
    need_gpu()
    lens = I.decode_lengths(64, 512, 8192, seed=21)
    q, k, v, table, sl = (t.cuda() for t in I.make_paged_decode(64, 64, 8, 128, 16, lens, seed=21))
    pages = k.shape[0]
    kc, vc = (torch.zeros(k.shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.zeros((pages, 8, 2, 16), dtype=torch.uint8, device="cuda")
    ident = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    fa.cache_append(k.view(1, pages * 16, 8, 128), v.view(1, pages * 16, 8, 128), kc, vc, ident,
                    torch.zeros(1, dtype=torch.int32, device="cuda"), kv_scale=sc)
    o, lse = fa.decode_paged_fp8(q, kc, vc, sc, table, sl)
    assert fa.last_device_status()[0] == 0
    for b in (0, 7, 21, 33, 50, 63):
        n = (int(sl[b]) + 15) // 16
        pg = table[b, :n].long()
        local = torch.arange(n, dtype=torch.int32).view(1, n)
        args = (q[b:b + 1].cpu(), kc[pg].cpu(), vc[pg].cpu(), sc[pg].cpu(), local, sl[b:b + 1].cpu())
        _check(args, o[b:b + 1], lse[b:b + 1], 1 / math.sqrt(128))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences_share_the_ranges(d):
    """More sequences than threads look them up, most of them short or empty, a few long: every way for a
    sequence to lie in the ranges (several in one, one in several, ending on a border)."""
    need_gpu()
    g = torch.Generator().manual_seed(15)
    lens = torch.randint(0, 40, (400,), generator=g).tolist()
    for b, n in ((0, 0), (7, 1500), (8, 128), (9, 640), (200, 2900), (399, 900)):
        lens[b] = n
    args = _make(400, 2, 1, d, 16, lens, seed=15)
    assert fa.decode_fp8_workspace_size(400, 2, 1, d, 16, args[4].shape[1]) > 0
    o, lse = _run(args, scale=0.1)
    _check(args, o, lse, 0.1)
    o, lse = _run(args, scale=0.1, window_left=300)
    _check(args, o, lse, 0.1, 300)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,d", [(6, 2, 128), (24, 2, 64)])
def test_a_batch_of_short_sequences_runs_whole(H, Hkv, d):
    need_gpu()
    g = torch.Generator().manual_seed(16)
    lens = torch.randint(0, 385, (150,), generator=g).tolist()
    args = _make(150, H, Hkv, d, 32, lens, seed=16, max_pages=12)
    assert fa.decode_fp8_workspace_size(150, H, Hkv, d, 32, 12) == 0
    o, lse = _run(args, scale=0.1)
    _check(args, o, lse, 0.1)


@pytest.mark.gpu
def test_given_outputs_and_their_checks():
    need_gpu()
    args = [t.cuda() for t in _make(2, 4, 2, 64, 8, [30, 9], seed=14)]
    want = fa.decode_paged_fp8(*args)
    o = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 4), 7.0, device="cuda")
    got = fa.decode_paged_fp8(*args, out=o, lse=lse)
    assert got[0] is o and got[1] is lse and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for kw in ({"out": o.float()}, {"out": o[:1]}, {"lse": lse.t()}, {"lse": lse.cpu()}, {"out": o[..., ::2]},
               {"workspace": torch.empty(8, dtype=torch.uint8)}, {"window_left": -1}, {"window_left": 0.5}):
        with pytest.raises((ValueError, TypeError)):
            fa.decode_paged_fp8(*args, **kw)
    with pytest.raises(fa.FAError):
        fa.decode_paged_fp8(*args, scale=-1.0)
