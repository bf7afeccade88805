"""The operators around the attention, without a GPU: the oracle's definitions
(oracle/serving.py) pinned to independent facts, and the refusals of the C entry
points and the Python binding.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_51_b200 as fa
import oracle
from exact_io_aware_51_b200 import build as fabuild
from exact_io_aware_51_b200 import inputs as I
from oracle import serving as S


@pytest.fixture(scope="module")
def L():
    fabuild.build()
    return fa.lib()


# ---------------------------------------------------------------- the oracle
def _tables(rows, d, seed=0):
    a = np.random.default_rng(seed).uniform(-4, 4, (rows, d // 2))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation_by_position(interleaved):
    """Scores of rotated q and k depend on the distance of their positions alone."""
    d, N = 64, 40
    ang = np.arange(N)[:, None] * 100.0 ** (-np.arange(0, d, 2) / d)
    cos, sin = np.cos(ang), np.sin(ang)
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, d))
    rows = np.broadcast_to(q, (1, N, 1, d)), np.broadcast_to(k, (1, N, 1, d))
    rq, rk = (S.norm_rope(x, None, cos, sin, interleaved=interleaved)[0, :, 0] for x in rows)
    s = rq @ rk.T
    for off in (0, 1, 7):
        assert np.allclose(np.diagonal(s, -off), s[off, 0], atol=1e-12)
    assert np.allclose(np.diagonal(s), q @ k, atol=1e-12)
    # the two pairings are one permutation of the features apart
    perm = np.concatenate([np.arange(0, d, 2), np.arange(1, d, 2)])
    a = S.norm_rope(rows[0], None, cos, sin, interleaved=True)[..., perm]
    b = S.norm_rope(rows[0][..., perm], None, cos, sin, interleaved=False)
    assert np.allclose(a, b, atol=1e-12)


def test_norm_equals_torch_rms_norm():
    x = torch.randn(2, 3, 4, 64, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
    w = torch.randn(64, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    cos, sin = np.ones((3, 32)), np.zeros((3, 32))
    ref = torch.nn.functional.rms_norm(x, (64,), w, 1e-6).numpy()
    assert np.allclose(S.norm_rope(x, w, cos, sin), ref, atol=1e-13)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_backward_by_central_differences(interleaved, norm):
    rng = np.random.default_rng(4)
    B, N, H, d = 2, 3, 2, 64
    x, g = rng.standard_normal((2, B, N, H, d))
    w = 1 + 0.3 * rng.standard_normal(d) if norm else None
    cos, sin = _tables(9, d)
    pos = np.array([[0, 8, -1], [3, 3, 5]])

    def loss(x, w):
        return np.sum(g * S.norm_rope(x, w, cos, sin, pos, 1e-3, interleaved))

    dx, dw = S.norm_rope_backward(x, w, cos, sin, g, pos, 1e-3, interleaved)
    assert np.all(dx[0, 2] == 0)
    h = 1e-6
    for idx in [(0, 0, 1, 3), (0, 1, 0, 63), (1, 2, 1, 32), (0, 2, 0, 5), (1, 0, 0, 31)]:
        e = np.zeros_like(x)
        e[idx] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[idx]) <= 1e-7
    if norm:
        for i in (0, 31, 32, 63):
            e = np.zeros(d)
            e[i] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) <= 1e-6


def test_e4m3_values_and_rounding_equal_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(S.e4m3_values(), ref, equal_nan=True)
    x = torch.randn(4096, generator=torch.Generator().manual_seed(5)) * torch.logspace(-4, 2, 4096)
    x = torch.cat([x, torch.tensor(ref[:127]).float(), torch.tensor((ref[:126] + ref[1:127]) / 2).float()])  # and every tie
    row = torch.cat([x.clamp(-448, 448), torch.tensor([448.0])])
    c, b = S.quantise_rows(row)
    assert b == 127
    assert np.array_equal(S.e4m3_values()[c], row.to(torch.float8_e4m3fn).float().double().numpy())


def test_quantised_rows_keep_the_formats_precision():
    """Every value comes back within half a step of e4m3 (2^-4 of it, or half the smallest
    step below the normal range), for any size of row; the scale is the smallest that fits."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((300, 64)) * 2.0 ** rng.uniform(-100, 100, (300, 1))
    c, b = S.quantise_rows(x)
    y = S.dequantise(c, b)
    s = 2.0 ** (b.astype(float) - 127)[:, None]
    assert np.all(np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10))
    amax = np.abs(x).max(-1)
    assert np.all(amax <= 448 * s[:, 0]) and np.all(amax > 224 * s[:, 0])
    c, b = S.quantise_rows(np.array([[0.0] * 64, [1.0] * 63 + [np.inf], [np.nan] + [0.0] * 63, [448.0] + [0.0] * 63,
                                     [np.nextafter(448.0, 500)] + [0.0] * 63, [2.0 ** -133] * 64]))
    assert list(b) == [1, 255, 255, 127, 128, 1]
    assert np.all(np.isnan(S.dequantise(c, b)[1:3])) and np.all(c[0] == 0)
    assert np.all(S.dequantise(c, b)[5] == 2.0 ** -133)


def test_paged_append_read_and_window_against_plain_slices():
    rng = np.random.default_rng(7)
    q, kc, vc, table, lens = I.make_paged_decode(3, 4, 2, 64, 8, [9, 0, 30], seed=3, spare_pages=1)
    table = table.clone()
    start, count = np.array([4, 0, 29]), np.array([5, 0, 1])
    k, v = rng.standard_normal((2, 3, 6, 2, 64))
    nk, nv, _ = S.cache_append(k, v, kc.float().numpy().astype(float), vc.float().numpy().astype(float), table, start, count=count)
    rk = S.cache_read(nk, table, lens, 32)
    old = S.cache_read(kc.float(), table, lens, 32)
    assert np.array_equal(rk[0, 4:9], k[0, :5]) and np.array_equal(rk[0, :4], old[0, :4])
    assert np.array_equal(rk[2, 29], k[2, 0]) and np.array_equal(rk[2, :29], old[2, :29])
    assert np.all(rk[0, 9:] == 0) and np.all(rk[1] == 0) and np.all(rk[2, 30:] == 0)
    # a window as long as the sequence is no window; a window of 0 returns the last V
    full, lse = oracle.decode_paged(q, nk, nv, table, lens, 0.125)
    for w in (None, 29, 1000):
        o, l = S.decode_window(q, nk, nv, table, lens, 0.125, w)
        assert np.allclose(o, full, atol=1e-12) and np.allclose(l[[0, 2]], lse[[0, 2]], atol=1e-12)
    o, _ = S.decode_window(q, nk, nv, table, lens, 0.125, 0)
    assert np.allclose(o[2], np.repeat(S.cache_read(nv, table, lens, 32)[2, 29], 2, axis=0))
    # a window of w positions before the last: softmax over the slice
    o, _ = S.decode_window(q, nk, nv, table, lens, 0.125, 10)
    s = 0.125 * rk[2, 19:30, 0] @ q[2, 0].double().numpy()
    p = np.exp(s - s.max())
    assert np.allclose(o[2, 0], p @ S.cache_read(nv, table, lens, 32)[2, 19:30, 0] / p.sum())


# ---------------------------------------------------------------- refusals of the C entry points
def test_norm_rope_validation(L):
    f, b = L.fa_qk_norm_rope, L.fa_qk_norm_rope_bwd

    def call(Q=16, K=16, wq=16, wk=16, c=16, s=16, pos=None, Qo=16, Ko=16, B=1, N=4, H=2, Hkv=2, d=64, qs=None, ks=None,
             rows=8, eps=1e-6, inter=0, dt=0, wdt=0):
        return f(Q, K, wq, wk, c, s, pos, Qo, Ko, B, N, H, Hkv, d, qs, ks, rows, eps, inter, dt, wdt, None)

    def back(wq=16, wk=16, gq=16, gk=16, dwq=16, dwk=16, N=4, H=2, gs=None, ws=256, size=1 << 20, dt=0, dq=16):
        return b(16, 16, wq, wk, 16, 16, None, gq, gk, dq, 16, dwq, dwk, 1, N, H, 2, 64, None, None, gs, None, 8, 1e-6, 0,
                 dt, 0, ws, size, None)

    assert call(d=96) == -2
    assert call(B=-1) == -1 and call(N=-1) == -1 and call(H=-1) == -1 and call(Hkv=-1) == -1
    assert call(dt=2) == -1 and call(wdt=2) == -1 and call(inter=2) == -1
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == -1
    assert call(wq=None) == -1 and call(wk=None) == -1            # both gains or none
    assert call(rows=3) == -1                                     # 4 positions, 3 rows in the tables
    assert call(rows=-1) == -1
    for name in ("Q", "K", "c", "s", "Qo", "Ko"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: 8}) == -3, name
    assert call(pos=2) == -3 and call(wq=8) == -3
    assert call(B=1 << 12, N=1 << 20, rows=1 << 21) == -8         # B * N beyond 2^31
    assert call(Hkv=65536) == -8
    st = (fa.ctypes.c_longlong * 3)(1024, 4, 64)
    assert call(qs=st) == -3 and call(ks=st) == -3                # strides of 8 bytes
    assert call(qs=st, dt=1, Q=8) == -3
    assert call(B=0) == 0 and call(N=0, Q=None, K=None) == 0 and call(H=0, Hkv=0) == 0
    # the backward
    assert back(wq=None) == -1 and back(dwq=None) == -1 and back(dwk=None) == -1
    assert back(gq=None) == -1 and back(gk=None) == -1
    assert back(gq=8) == -3 and back(dwq=8) == -3 and back(gs=st) == -3
    need = L.fa_qk_norm_rope_workspace_size(64)
    assert need > 0 and need % 256 == 0 and L.fa_qk_norm_rope_workspace_size(96) == 0
    assert back(ws=None) == -4 and back(size=need - 1) == -4 and back(ws=272) == -4
    assert back(dq=8) == -3
    assert back(wq=None, wk=None, dwq=None, dwk=None, N=0, ws=None, size=0) == 0


def test_norm_rope_limits(L):
    """The limits that the header states, from both sides (the pointers are refused next)."""
    def call(B=1, N=4, H=2, Hkv=2, rows=1 << 23):
        return L.fa_qk_norm_rope(None, None, None, None, None, None, None, None, None, B, N, H, Hkv, 64, None, None, rows,
                                 0.0, 0, 0, 0, None)

    for size, most in (("B", 65535), ("H", 65535), ("Hkv", 65535), ("N", 1 << 22)):
        assert call(**{size: most}) == -1 and call(**{size: most + 1}) == -8, size
    assert call(B=511, N=1 << 22) == -1 and call(B=512, N=1 << 22) == -8                      # B * N < 2^31
    for size in ("H", "Hkv"):                                                                  # 2^40 elements
        assert call(N=1 << 22, **{size: 4095}) == -1 and call(N=1 << 22, **{size: 4096}) == -8


def test_cache_validation(L):
    def append(K=16, V=16, kc=16, vc=16, sc=16, bt=16, st=16, ct=None, B=2, N=3, Hkv=2, d=64, ks=None, vs=None, P=16,
               npg=10, mp=4, fp8=1):
        return L.fa_cache_append(K, V, kc, vc, sc, bt, st, ct, B, N, Hkv, d, ks, vs, P, npg, mp, fp8, None)

    def read(kc=16, vc=16, sc=16, bt=16, sl=16, K=16, V=16, B=2, N=3, Hkv=2, d=64, P=16, npg=10, mp=4, fp8=1):
        return L.fa_cache_read(kc, vc, sc, bt, sl, K, V, B, N, Hkv, d, P, npg, mp, fp8, None)

    for f in (append, read):
        assert f(d=96) == -2
        for P in (0, 4, 12, 8192):
            assert f(P=P) == -2, P
        assert f(B=-1) == -1 and f(N=-1) == -1 and f(Hkv=0) == -1 and f(npg=0) == -1 and f(mp=0) == -1 and f(fp8=2) == -1
        assert f(npg=1 << 27) == -8 and f(mp=(1 << 26) + 1) == -8 and f(B=65536) == -8 and f(Hkv=65536) == -8
        assert f(B=65535, N=1 << 24, Hkv=64) == -8 and f(N=(1 << 30) + 1) == -8
        for name in ("K", "V", "kc", "vc", "sc", "bt"):
            assert f(**{name: None}) == -1, name
        for name in ("K", "V", "kc", "vc", "sc"):
            assert f(**{name: 8}) == -3, name
        assert f(bt=2) == -3
        assert f(B=0) == 0 and f(N=0, K=None, V=None) == 0
    assert append(st=None) == -1 and read(sl=None) == -1 and append(st=2) == -3 and append(ct=2) == -3
    bad = (fa.ctypes.c_longlong * 3)(1024, 64, 4)
    assert append(ks=bad) == -3 and append(vs=bad) == -3


def test_decode_fp8_validation(L):
    def call(ptr=16, q=None, sc=16, B=2, H=8, Hkv=2, d=128, P=16, npg=10, mp=4, scale=0.1, w=-1, ws=None, size=0):
        q = ptr if q is None else q
        return L.fa_decode_paged_fp8(q, ptr, ptr, sc, ptr, ptr, ptr, ptr, B, H, Hkv, d, P, npg, mp, scale, w, ws, size,
                                     None)

    assert call(ptr=None) == -1 and call(sc=None) == -1
    assert call(d=96) == -2 and call(P=24) == -2 and call(P=4) == -2 and call(Hkv=3) == -1
    assert call(scale=0.0) == -1 and call(scale=float("nan")) == -1 and call(w=-2) == -1
    assert call(npg=0) == -1 and call(mp=0) == -1 and call(B=-1) == -1
    assert call(npg=1 << 28) == -8 and call(mp=(1 << 26) + 1) == -8 and call(B=65536) == -8
    assert call(B=256, mp=1 << 26) == -8                          # 2^38 positions in all
    assert call(q=8) == -3 and call(sc=8) == -3
    assert call(ws=8, size=64) == -4
    assert call(B=0, ptr=None) == 0
    size = L.fa_decode_fp8_workspace_size
    assert size(64, 64, 8, 128, 16, 8, -1) == 0                   # a full batch of short sequences
    n = size(1, 32, 8, 128, 16, 4096, -1)
    assert n > 0 and n % 256 == 0
    assert 0 <= size(1, 32, 8, 128, 16, 4096, 127) < n            # a window needs fewer chunks
    assert size(1, 32, 8, 96, 16, 4096, -1) == 0 and size(1, 32, 8, 128, 16, 4096, -2) == 0


# ---------------------------------------------------------------- the binding's build
def test_binding_belongs_to_one_pytorch(L, monkeypatch):
    """Under another PyTorch than it was compiled against it counts as out of date, and is not loaded."""
    kc = torch.zeros(5, 8, 2, 64, dtype=torch.bfloat16)
    bt, st = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    assert fabuild.up_to_date()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    monkeypatch.setattr(fa, "_BINDING", None)
    assert not fabuild.up_to_date()
    with pytest.raises(fa.FAError, match="another PyTorch"):
        fa.cache_read(kc, kc, bt, st, 4)
    monkeypatch.undo()
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_read(kc, kc, bt, st, 4)


def test_libraries_are_linked_where_the_binding_fails(tmp_path, monkeypatch):
    """A C user needs no binding: what goes wrong with it is raised after the libraries are there."""
    libs = {n: tmp_path / f"{n.lower()}.so" for n in ("LIB", "PROBE_LIB", "DEBUG_LIB")}
    for n, p in libs.items():
        monkeypatch.setattr(fabuild, n, p)
    monkeypatch.setattr(fabuild, "BUILD", tmp_path / "_build")
    monkeypatch.setattr(fabuild, "_compile", lambda src, verbose, debug=False: tmp_path / f"{src.stem}{debug}.o")

    def linker(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        assert "-shared" in cmd and all(x.endswith(".o") for x in cmd[cmd.index("-o") + 2:-2])
        open(out, "w").close()
        return fabuild.subprocess.CompletedProcess(cmd, 0, "", "")

    def broken(verbose):
        raise RuntimeError("no compiler for the binding")

    monkeypatch.setattr(fabuild, "subprocess", type("S", (), {"run": staticmethod(linker),
                                                              "CompletedProcess": fabuild.subprocess.CompletedProcess}))
    monkeypatch.setattr(fabuild, "_binding", broken)
    with pytest.raises(RuntimeError, match="no compiler"):
        fabuild.build(force=True)
    assert all(p.exists() for p in libs.values())


# ---------------------------------------------------------------- refusals of the binding
def test_python_norm_rope_refusals(L):
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(8, 32)
    w = torch.zeros(64, dtype=torch.bfloat16)
    f = fa.qk_norm_rope
    with pytest.raises(ValueError, match="CUDA"):
        f(q, k, c, c)
    for bad in ((q[0], k, c, c), (q, k[:1], c, c), (q, k[..., :32], c, c), (q, k, c[:, :16], c[:, :16]), (q, k, c, c[:4]),
                (q, k, c[:2], c[:2]), (q, k, c[:, ::2].repeat(1, 2)[:, ::2], c)):
        with pytest.raises(ValueError):
            f(*bad)
    for bad in ((q.half(), k, c, c), (q, k.float(), c, c), (q, k, c.double(), c)):
        with pytest.raises(TypeError):
            f(*bad)
    with pytest.raises(ValueError, match="both gains"):
        f(q, k, c, c, q_weight=w)
    with pytest.raises(ValueError):
        f(q, k, c, c, q_weight=w[:32], k_weight=w[:32])
    with pytest.raises(TypeError):
        f(q, k, c, c, q_weight=w, k_weight=w.float())
    with pytest.raises(TypeError):
        f(q, k, c, c, positions=torch.zeros(2, 3, dtype=torch.int64))
    with pytest.raises(ValueError):
        f(q, k, c, c, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="tensor"):
        f(q, None, c, c)
    with pytest.raises(TypeError):
        f(q, k, c, c, eps="small")
    with pytest.raises(RuntimeError, match="ambiguous"):
        f(q, k, c, c, interleaved=torch.ones(2))


def test_forward_mode_derivatives_are_refused(L):
    """There is none, and a tangent must not be lost: fa.attention refuses it, too."""
    import torch.autograd.forward_ad as fwad

    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    c, w = torch.zeros(8, 32), torch.zeros(64, dtype=torch.bfloat16)
    given = {"q": q, "k": k, "cos": c, "sin": c, "q_weight": w, "k_weight": w}
    with fwad.dual_level():
        for name, t in given.items():
            args = {**given, name: fwad.make_dual(t, torch.ones_like(t))}
            with pytest.raises(NotImplementedError, match="forward-mode"):
                fa.qk_norm_rope(**args)
            with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
                fa.qk_norm_rope(**args)
            with pytest.raises(ValueError, match="CUDA"), fwad._set_fwd_grad_enabled(False):
                fa.qk_norm_rope(**args)
        with pytest.raises(ValueError, match="CUDA"):
            fa.qk_norm_rope(**given)


def test_python_cache_refusals(L):
    kc = torch.zeros(5, 8, 2, 64, dtype=torch.uint8)
    sc = torch.zeros(5, 2, 2, 8, dtype=torch.uint8)
    bt = torch.zeros(3, 2, dtype=torch.int32)
    st = torch.zeros(3, dtype=torch.int32)
    k = torch.zeros(3, 1, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_append(k, k, kc, kc, bt, st, kv_scale=sc)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_read(kc, kc, bt, st, 4, kv_scale=sc)
    with pytest.raises(ValueError, match="CUDA"):
        fa.decode_paged_fp8(q, kc, kc, sc, bt, st)
    with pytest.raises(ValueError, match="kv_scale"):
        fa.cache_read(kc, kc, bt, st, 4)
    with pytest.raises(ValueError, match="kv_scale"):
        fa.cache_read(kc, kc, bt, st, 4, kv_scale=sc[:, :, :1])
    with pytest.raises(ValueError, match="takes no kv_scale"):
        fa.cache_read(kc.bfloat16(), kc.bfloat16(), bt, st, 4, kv_scale=sc)
    with pytest.raises(TypeError):
        fa.cache_read(kc.float(), kc.float(), bt, st, 4)
    with pytest.raises(TypeError):
        fa.cache_read(kc, kc, bt.long(), st, 4, kv_scale=sc)
    with pytest.raises(TypeError):
        fa.cache_read(kc, kc, bt, st, 4, kv_scale=sc.float())
    with pytest.raises(ValueError):
        fa.cache_read(kc, kc, bt, st[:2], 4, kv_scale=sc)
    with pytest.raises(ValueError, match="contiguous"):
        fa.cache_read(kc.transpose(1, 2).contiguous().transpose(1, 2), kc, bt, st, 4, kv_scale=sc)
    with pytest.raises(TypeError):
        fa.decode_paged_fp8(q, kc.bfloat16(), kc.bfloat16(), None, bt, st)
    for name, fn in (("CUDA", fa.cache_append),):
        with pytest.raises(ValueError, match=name):
            fn(k, k, kc.bfloat16(), kc.bfloat16(), bt, st)


def test_rope_tables_hold_far_angles():
    """cos and sin of positions up to 2^20 to fp32 rounding (a float32 angle would be off by up to 2^-4)."""
    n = 1 << 20
    cos, sin = fa.rope_tables(n, 64, device="cpu")
    assert cos.shape == (n, 32) and cos.dtype == torch.float32
    p, i = n - 1, 1
    a = p * 10000.0 ** (-2 * i / 64)
    assert abs(float(cos[p, i]) - np.cos(a)) <= 2.0 ** -24 + 1e-9 and abs(float(sin[p, i]) - np.sin(a)) <= 2.0 ** -24 + 1e-9
    assert torch.allclose(cos * cos + sin * sin, torch.ones(()), atol=4 * 2.0 ** -24)
