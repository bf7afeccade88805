"""Writing and reading a paged cache: exact against the oracle.

The 8-bit format has no freedom (a power-of-two scale, x / scale exact, one
rounding to the nearest code), so codes, scale bytes and everything that was
not to be written are compared bit by bit; so are the rows read back, code *
scale rounded once to bf16.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_51_b200 as fa
from oracle import serving as S
from tests.helpers import need_gpu


def _table(need, page, spare, width, g):
    n = [(x + page - 1) // page for x in need]
    total = sum(n) + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(n), max([width] + n)), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(n):
        table[b, :k] = order[at:at + k]
        at += k
    return table, total


def _pool(pages, page, Hkv, d, fp8, g):
    shape = (pages, page, Hkv, d)
    if fp8:
        kc, vc = (torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in range(2))
        return kc, vc, torch.randint(0, 256, (pages, Hkv, 2, page), generator=g, dtype=torch.uint8)
    return *(torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2)), None


def _rows(shape, g):
    """Rows of very different sizes, bf16."""
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-12, 12, (*shape[:-1], 1), generator=g).float())
    return x.to(torch.bfloat16)


CASES = [
    # fp8, B, N, Hkv, d, page, starts, counts, packed
    (True, 3, 1, 8, 128, 16, [0, 15, 16], None, False),
    (True, 2, 37, 3, 64, 8, [5, 0], [37, 11], True),
    (True, 2, 130, 1, 128, 64, [1, 63], [130, 0], False),
    (True, 4, 9, 5, 64, 4096, [0, 4095, 100, 8000], [9, 9, 1, 5], True),
    (True, 1, 300, 2, 128, 32, [7], None, True),
    (False, 3, 1, 4, 64, 16, [0, 31, 32], None, False),
    (False, 2, 41, 3, 128, 8, [3, 0], [40, 7], True),
]


def _name(c):
    return f"{'fp8' if c[0] else 'bf16'}-B{c[1]}N{c[2]}kv{c[3]}d{c[4]}P{c[5]}"


def _make(case, seed):
    fp8, B, N, Hkv, d, page, starts, counts, packed = case
    g = torch.Generator().manual_seed(seed)
    counts_ = [N] * B if counts is None else counts
    table, pages = _table([s + c for s, c in zip(starts, counts_)], page, 2, 3, g)
    kc, vc, sc = _pool(pages, page, Hkv, d, fp8, g)
    if packed:
        x = _rows((B, N, 2 + 2 * Hkv, d), g).cuda()
        k, v = x[:, :, 2:2 + Hkv], x[:, :, 2 + Hkv:]
    else:
        k, v = _rows((B, N, Hkv, d), g).cuda(), _rows((B, N, Hkv, d), g).cuda()
    start = torch.tensor(starts, dtype=torch.int32)
    count = None if counts is None else torch.tensor(counts, dtype=torch.int32)
    return k, v, kc, vc, sc, table, start, count


def _np(t):
    return None if t is None else (t.double().numpy() if t.dtype == torch.bfloat16 else t.numpy())


def _c(t):
    return None if t is None else t.cuda()


def _same_pool(got, ref, fp8):
    a = got.cpu()
    assert np.array_equal(a.numpy() if fp8 else a.double().numpy(), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=_name)
def test_append_and_read_match_oracle(case):
    need_gpu()
    fp8, B, N, Hkv, d, page = case[:6]
    k, v, kc, vc, sc, table, start, count = _make(case, seed=31)
    rk, rv, rs = S.cache_append(k.cpu().double(), v.cpu().double(), _np(kc), _np(vc), table, start, _np(sc), count)
    gk, gv, gs = kc.cuda(), vc.cuda(), _c(sc)
    assert fa.cache_append(k, v, gk, gv, table.cuda(), start.cuda(), kv_scale=gs, count=_c(count)) is None
    assert fa.last_device_status()[0] == 0
    _same_pool(gk, rk, fp8)
    _same_pool(gv, rv, fp8)
    if fp8:
        assert np.array_equal(gs.cpu().numpy(), rs)
    # read back: the appended length, a length past every end, and one position
    lens = start + (N if count is None else count)
    K, V = S.dequantise_cache(rk, rv, rs) if fp8 else (rk, rv)
    for length in (int(lens.max()) + 3, 1):
        out = fa.cache_read(gk, gv, table.cuda(), lens.cuda(), length, kv_scale=gs)
        for got, pool in zip(out, (K, V)):
            ref = torch.from_numpy(S.cache_read(pool, table, lens, length)).to(torch.bfloat16)
            assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=12345.0),
                               torch.nan_to_num(ref.float(), nan=12345.0))
    assert fa.last_device_status()[0] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rows_at_the_formats_edges(d):
    """Zero rows, subnormals, the largest bf16, rows on each side of a power of two's 448, every tie, Inf and NaN."""
    need_gpu()
    vals = torch.from_numpy(S.e4m3_values()[:127]).float()
    ties = (vals[1:] + vals[:-1]) / 2
    big = torch.finfo(torch.bfloat16).max
    heads = [torch.zeros(d), torch.full((d,), 2.0 ** -133), torch.full((d,), -2.0 ** -126), torch.full((d,), big),
             torch.cat([vals, vals[-1:]])[-d:], torch.cat([torch.tensor([448.0, 448.0]), ties])[:d],
             torch.cat([torch.tensor([448.0, 448.0]), -ties])[-d:], torch.linspace(-448, 448, d), torch.linspace(-450, 450, d),
             torch.linspace(-1, 1, d) * 2.0 ** -120, torch.full((d,), -0.0)]
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = torch.linspace(-2, 2, d)
        x[d // 3] = bad
        heads.append(x)
    rows = torch.stack(heads).to(torch.bfloat16).reshape(1, 1, len(heads), d)
    Hkv, page = len(heads), 8
    kc = torch.zeros((1, page, Hkv, d), dtype=torch.uint8)
    sc = torch.zeros((1, Hkv, 2, page), dtype=torch.uint8)
    table, start = torch.zeros((1, 1), dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    v = rows.flip(2)
    rk, rv, rs = S.cache_append(rows.double(), v.double(), kc.numpy(), kc.numpy(), table, start, sc.numpy())
    gk, gv, gs = kc.cuda(), kc.clone().cuda(), sc.cuda()
    fa.cache_append(rows.cuda(), v.cuda(), gk, gv, table.cuda(), start.cuda(), kv_scale=gs)
    assert np.array_equal(gs.cpu().numpy(), rs)
    finite = rs[0, :, 0, 3] != 255
    assert np.array_equal(gk.cpu().numpy()[0, 3][finite], rk[0, 3][finite])
    assert np.all(gk.cpu().numpy()[0, 3][~finite] & 127 == 127)      # NaN codes
    out, _ = fa.cache_read(gk, gv, table.cuda(), start.cuda() + 1, 4, kv_scale=gs)
    ref = torch.from_numpy(S.dequantise_cache(rk, rv, rs)[0][0, 3]).to(torch.bfloat16)
    got = out[0, 3].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)) and bool((torch.isnan(got).any(-1).numpy() == ~finite).all())
    assert torch.equal(got[torch.from_numpy(finite)], ref[torch.from_numpy(finite)])


@pytest.mark.gpu
def test_float8_tensors_and_codes_are_one_format():
    need_gpu()
    case = (True, 2, 20, 2, 64, 16, [0, 9], None, False)
    k, v, kc, vc, sc, table, start, _ = _make(case, seed=32)
    a = [t.cuda() for t in (kc, vc, sc)]
    b = [kc.cuda().view(torch.float8_e4m3fn), vc.cuda().view(torch.float8_e4m3fn), sc.cuda().view(torch.float8_e8m0fnu)]
    for x in (a, b):
        fa.cache_append(k, v, x[0], x[1], table.cuda(), start.cuda(), kv_scale=x[2])
    for x, y in zip(a, b):
        assert torch.equal(x, y.view(torch.uint8))
    lens = start.cuda() + 20
    for x, y in zip(fa.cache_read(a[0], a[1], table.cuda(), lens, 29, kv_scale=a[2]),
                    fa.cache_read(b[0], b[1], table.cuda(), lens, 29, kv_scale=b[2])):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    # the scale bytes are the values of torch's 8-bit exponent type
    pos = int(start[1])
    pg = int(table[1, pos // 16])
    row = a[0][pg, pos % 16, 1].view(torch.float8_e4m3fn).float() * b[2][pg, 1, 0, pos % 16].float()
    assert torch.equal(row, fa.cache_read(a[0], a[1], table.cuda(), lens, 29, kv_scale=a[2])[0][1, pos, 1].float())


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_bad_device_data_is_reported_and_left_out(fp8):
    need_gpu()
    case = (fp8, 3, 12, 2, 64, 8, [4, 0, 9], [12, 5, 7], False)
    k, v, kc, vc, sc, table, start, count = _make(case, seed=33)
    pages = kc.shape[0]

    def append(table, start, count):
        pools = [kc.cuda(), vc.cuda(), _c(sc)]
        fa.last_device_status()
        fa.cache_append(k, v, pools[0], pools[1], table.cuda(), start.cuda(), kv_scale=pools[2], count=count.cuda())
        return pools, fa.last_device_status()

    def expect(b_out, table, pools, skip=()):
        c = count.clone()
        c[b_out] = 0
        ref = S.cache_append(k.cpu().double(), v.cpu().double(), _np(kc), _np(vc), table, start, _np(sc), c)
        got = [p if p is None else p.cpu() for p in pools]
        for g, r in zip(got, ref):
            if r is not None:
                assert np.array_equal(g.numpy() if fp8 else g.double().numpy(), r)

    for what, value in (("start", -1), ("start", table.shape[1] * 8 - 11), ("count", 13), ("count", -1)):
        s, c = start.clone(), count.clone()
        (s if what == "start" else c)[0] = value
        pools, (rc, detail) = append(table, s, c)
        assert rc == -9 and detail == 0x2000 | 0xD1, (what, value)
        expect(0, table, pools)
    for page in (pages, -5):
        t = table.clone()
        t[1, 0] = page
        pools, (rc, detail) = append(t, start, count)
        assert rc == -9 and detail == 0x2000 | 0xD2
        expect(1, table, pools)
    # reads: a bad length gives zeros, a bad page zeros for its positions
    lens = (start + count).cuda()
    pools = [kc.cuda(), vc.cuda(), _c(sc)]
    clean = fa.cache_read(*pools[:2], table.cuda(), lens, 20, kv_scale=pools[2])
    for bad in (-1, table.shape[1] * 8 + 1):
        l2 = lens.clone()
        l2[2] = bad
        out = fa.cache_read(*pools[:2], table.cuda(), l2, 20, kv_scale=pools[2])
        assert fa.last_device_status()[0] == -9
        assert torch.count_nonzero(out[0][2].view(torch.int16)) == 0
        assert torch.equal(out[0][:2].view(torch.int16), clean[0][:2].view(torch.int16))
    t = table.clone()
    t[0, 1] = pages + 7
    out = fa.cache_read(*pools[:2], t.cuda(), lens, 20, kv_scale=pools[2])
    assert fa.last_device_status() == (-9, 0x2000 | 0xD2)
    assert torch.count_nonzero(out[1][0, 8:16].view(torch.int16)) == 0
    assert torch.equal(out[1][0, :8].view(torch.int16), clean[1][0, :8].view(torch.int16))
    assert fa.last_device_status()[0] == 0


@pytest.mark.gpu
def test_table_entries_past_the_end_are_not_read():
    """A table holds what it likes behind a sequence's last page, and padded rows what they like."""
    need_gpu()
    case = (True, 2, 10, 2, 64, 8, [0, 3], [4, 10], False)
    k, v, kc, vc, sc, table, start, count = _make(case, seed=34)
    k, v = k.clone(), v.clone()
    k[0, 4:], v[0, 4:] = float("nan"), float("nan")
    gk, gv, gs = kc.cuda(), vc.cuda(), sc.cuda()
    wide = torch.full((2, 8), 2 ** 30, dtype=torch.int32)
    wide[0, :1], wide[1, :2] = table[0, :1], table[1, :2]
    fa.cache_append(k, v, gk, gv, wide.cuda(), start.cuda(), kv_scale=gs, count=count.cuda())
    fa.cache_read(gk, gv, wide.cuda(), (start + count).cuda(), 64, kv_scale=gs)
    assert fa.last_device_status()[0] == 0
    ref = S.cache_append(k.nan_to_num(0).cpu().double(), v.nan_to_num(0).cpu().double(), _np(kc), _np(vc), table, start, _np(sc), count)
    assert np.array_equal(gk.cpu().numpy(), ref[0]) and np.array_equal(gs.cpu().numpy(), ref[2])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8,d", [(True, 128), (True, 64), (False, 128)])
def test_large_append(fp8, d):
    """Enough rows that a warp takes several groups of positions: sampled rows against the oracle, all other rows of
    the pools as they were, and the rows read back against the rows given."""
    need_gpu()
    B, N, Hkv, page = 8, 4096, 8, 16
    g = torch.Generator().manual_seed(36)
    starts = torch.randint(0, 50, (B,), generator=g).tolist()
    counts = [0, 1, N, N - 1, 5, 17, 2048, 3000]
    table, pages = _table([s + c for s, c in zip(starts, counts)], page, 3, 3, g)
    kc, vc, sc = _pool(pages, page, Hkv, d, fp8, g)
    k, v = _rows((B, N, Hkv, d), g), _rows((B, N, Hkv, d), g)
    gk, gv, gs = kc.cuda(), vc.cuda(), _c(sc)
    start, count = (torch.tensor(x, dtype=torch.int32) for x in (starts, counts))
    fa.cache_append(k.cuda(), v.cuda(), gk, gv, table.cuda(), start.cuda(), kv_scale=gs, count=count.cuda())
    assert fa.last_device_status()[0] == 0
    gk, gv, gs = gk.cpu(), gv.cpu(), None if gs is None else gs.cpu()
    written = torch.zeros((pages, page), dtype=torch.bool)
    for b in range(B):
        at = torch.arange(starts[b], starts[b] + counts[b])
        written[table[b, at // page].long(), at % page] = True
    assert torch.equal(gk[~written], kc[~written]) and torch.equal(gv[~written], vc[~written])
    if fp8:
        keep = ~written[:, None, None, :].expand(pages, Hkv, 2, page)
        assert torch.equal(gs[keep], sc[keep])
    for b in range(B):
        for n in {0, 1, counts[b] // 2, counts[b] - 9, counts[b] - 2, counts[b] - 1}:
            if not 0 <= n < counts[b]:
                continue
            pg, slot = int(table[b, (starts[b] + n) // page]), (starts[b] + n) % page
            for which, (x, pool) in enumerate(((k, gk), (v, gv))):
                if fp8:
                    codes, byte = S.quantise_rows(x[b, n].double())
                    assert np.array_equal(pool[pg, slot].numpy(), codes)
                    assert np.array_equal(gs[pg, :, which, slot].numpy(), byte)
                else:
                    assert torch.equal(pool[pg, slot], x[b, n])
    out = fa.cache_read(gk.cuda(), gv.cuda(), table.cuda(), (start + count).cuda(), N + 50, kv_scale=_c(gs))
    for x, y in zip((k, v), out):
        for b in range(B):
            got = y[b, starts[b]:starts[b] + counts[b]].cpu().float()
            ref = x[b, :counts[b]].float()
            top = ref.abs().amax(-1, keepdim=True)  # a code is off by 2^-4 of itself, or half the smallest step: 2^-10 of 448ths
            assert bool(((got - ref).abs() <= (torch.maximum(ref.abs() * 2.0 ** -4, top * 2.0 ** -17) if fp8 else 0 * top)).all())


@pytest.mark.gpu
def test_pools_beyond_32_bit_offsets():
    """Pools of 5 GB each (K, V), the sequences' pages at their far end: append, read and decode."""
    need_gpu()
    P, Hkv, d = 16, 8, 128
    pages = 5 * 2 ** 30 // (P * Hkv * d)
    kc, vc = (torch.empty((pages, P, Hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.empty((pages, Hkv, 2, P), dtype=torch.uint8, device="cuda")
    assert kc.numel() > 2 ** 32 and sc.numel() > 2 ** 25
    g = torch.Generator().manual_seed(35)
    table = (pages - 1 - torch.arange(6, dtype=torch.int32)).view(2, 3).cuda()
    k, v = _rows((2, 40, Hkv, d), g).cuda(), _rows((2, 40, Hkv, d), g).cuda()
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    fa.cache_append(k, v, kc, vc, table, start, kv_scale=sc)
    lens = torch.tensor([40, 33], dtype=torch.int32, device="cuda")
    near = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)  # the same rows in small pools
    small = [torch.zeros((6, P, Hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ssc = torch.zeros((6, Hkv, 2, P), dtype=torch.uint8, device="cuda")
    fa.cache_append(k, v, *small, near, start, kv_scale=ssc)
    for a, b in zip(fa.cache_read(kc, vc, table, lens, 40, kv_scale=sc), fa.cache_read(*small, near, lens, 40, kv_scale=ssc)):
        assert torch.equal(a, b) and torch.count_nonzero(a[0, 39]) > 0
    q = torch.randn((2, 16, d), generator=g).to(torch.bfloat16).cuda()
    for a, b in zip(fa.decode_paged_fp8(q, kc, vc, sc, table, lens), fa.decode_paged_fp8(q, *small, ssc, near, lens)):
        assert torch.equal(a, b)
    assert fa.last_device_status()[0] == 0


@pytest.mark.gpu
def test_empty_calls():
    need_gpu()
    kc = torch.zeros((2, 8, 2, 64), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((2, 2, 2, 8), dtype=torch.uint8, device="cuda")
    for B, N in ((0, 3), (2, 0)):
        k = torch.zeros((B, N, 2, 64), dtype=torch.bfloat16, device="cuda")
        bt = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
        st = torch.zeros((B,), dtype=torch.int32, device="cuda")
        fa.cache_append(k, k, kc, kc, bt, st, kv_scale=sc)
        out = fa.cache_read(kc, kc, bt, st, N, kv_scale=sc)
        assert out[0].shape == (B, N, 2, 64)
    assert torch.count_nonzero(kc) == 0
