"""Plain fp64 CPU oracle of the operators around the attention (TEST INFRASTRUCTURE ONLY).

Norm and rotation of query and key heads, the 8-bit row format of the paged
cache, writing and reading a paged cache, and decode with a window: the
definitions of ``include/fa.h`` written out in numpy float64.  Shares no code
with the CUDA path.

* For one row x with gain w:  r = 1 / sqrt(mean(x^2) + eps),  y = x r w, and each
  pair of features (a, b), read as the complex number a + b i, is multiplied by
  the position's cos + i sin.  Pairs are (i, i + d/2) or (2i, 2i + 1).
* Backward: the rotation by the opposite angle gives gr; dw = sum gr x r,
  dx = r w gr - x r^3 / d sum(w gr x).
* e4m3: sign, 4 exponent bits with bias 7, 3 fraction bits; the codes 0x7f and
  0xff are NaN, there is no infinity, the largest value is 448.
"""

from __future__ import annotations

import numpy as np

from .attention import _f64, _to_numpy, kv_head, forward_rows_head, paged_rows


def _pairs(x, interleaved):
    d = x.shape[-1]
    if interleaved:
        return x[..., 0:d:2] + 1j * x[..., 1:d:2]
    return x[..., :d // 2] + 1j * x[..., d // 2:]


def _from_pairs(z, interleaved):
    out = np.empty(z.shape[:-1] + (2 * z.shape[-1],))
    if interleaved:
        out[..., 0::2], out[..., 1::2] = z.real, z.imag
    else:
        out[..., :z.shape[-1]], out[..., z.shape[-1]:] = z.real, z.imag
    return out


def _angles(x, cos, sin, positions):
    """e^(i angle) [B, N, 1, d/2] of every row, 0 for padding (a negative position)."""
    B, N = x.shape[:2]
    z = _f64(_to_numpy(cos)) + 1j * _f64(_to_numpy(sin))
    pos = np.broadcast_to(np.arange(N), (B, N)) if positions is None else np.asarray(_to_numpy(positions), np.int64)
    rot = z[np.maximum(pos, 0)] * (pos >= 0)[..., None]
    return rot[:, :, None, :]


def norm_rope(x, w, cos, sin, positions=None, eps=1e-6, interleaved=False):
    """x [B, N, heads, d], w [d] or None (no norm) -> float64 of x's shape."""
    x = _f64(_to_numpy(x))
    y = x
    if w is not None:
        y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * _f64(_to_numpy(w))
    return _from_pairs(_pairs(y, interleaved) * _angles(x, cos, sin, positions), interleaved)


def norm_rope_backward(x, w, cos, sin, g, positions=None, eps=1e-6, interleaved=False):
    """(dx, dw) of sum(g * norm_rope(x, w, ...)); dw None without a norm."""
    x, g = _f64(_to_numpy(x)), _f64(_to_numpy(g))
    gr = _from_pairs(_pairs(g, interleaved) * np.conj(_angles(x, cos, sin, positions)), interleaved)
    if w is None:
        return gr, None
    w = _f64(_to_numpy(w))
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    dw = np.sum(gr * x * r, axis=(0, 1, 2))
    dx = r * w * gr - x * r ** 3 / x.shape[-1] * np.sum(w * gr * x, axis=-1, keepdims=True)
    return dx, dw


def e4m3_values() -> np.ndarray:
    """The 256 values of the e4m3 codes (NaN for 0x7f and 0xff)."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = (f / 8.0) * 2.0 ** -6 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)
        if c & 127 == 127:
            v = np.nan
        out[c] = -v if c & 128 else v
    return out


def quantise_rows(x):
    """(codes, scale bytes) of rows x [..., d]: e the smallest integer >= -126 with
    max|x| <= 448 * 2^e, byte e + 127, codes x / 2^e to the nearest value, ties to the
    even code.  A row with an Inf or NaN: byte 255, NaN codes."""
    x = _f64(_to_numpy(x))
    flat = x.reshape(-1, x.shape[-1])
    values = e4m3_values()[:127]  # the non-negative finite values, ascending; the code is the index
    codes = np.zeros(flat.shape, np.uint8)
    byte = np.zeros(flat.shape[0], np.uint8)
    for i, row in enumerate(flat):
        if not np.all(np.isfinite(row)):
            codes[i], byte[i] = 0x7F, 255
            continue
        amax = np.max(np.abs(row))
        e = -126
        while amax > 448.0 * 2.0 ** e:
            e += 1
        byte[i] = e + 127
        y = np.abs(row) / 2.0 ** e
        hi = np.clip(np.searchsorted(values, y), 1, 126)
        lo = hi - 1
        dl, dh = y - values[lo], values[hi] - y
        c = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
        codes[i] = c | np.where(np.signbit(row), 128, 0).astype(np.uint8)
    return codes.reshape(x.shape), byte.reshape(x.shape[:-1])


def dequantise(codes, scale_bytes):
    """float64 values of codes [..., d] with a scale byte per row."""
    b = np.asarray(_to_numpy(scale_bytes), np.float64)
    s = np.where(b == 255, np.nan, 2.0 ** (b - 127))
    return e4m3_values()[np.asarray(_to_numpy(codes), np.uint8)] * s[..., None]


def dequantise_cache(k_codes, v_codes, kv_scale):
    """(K, V) float64 [num_pages, page_size, Hkv, d] of an 8-bit paged cache (kv_scale [num_pages, Hkv, 2, page_size])."""
    s = np.moveaxis(np.asarray(_to_numpy(kv_scale), np.uint8), (1, 3), (3, 1))  # [pages, page_size, 2, Hkv]
    return dequantise(k_codes, s[:, :, 0]), dequantise(v_codes, s[:, :, 1])


def cache_append(k, v, k_cache, v_cache, block_table, start, kv_scale=None, count=None):
    """Copies of (k_cache, v_cache, kv_scale) with the new rows written: row n of sequence b at position
    start[b] + n.  numpy arrays; with kv_scale the pools hold codes (uint8), without it values (float64)."""
    k, v = _f64(_to_numpy(k)), _f64(_to_numpy(v))
    kc, vc = np.array(_to_numpy(k_cache)), np.array(_to_numpy(v_cache))
    sc = None if kv_scale is None else np.array(_to_numpy(kv_scale))
    table = np.asarray(_to_numpy(block_table), np.int64)
    start = np.asarray(_to_numpy(start), np.int64)
    B, N = k.shape[:2]
    count = np.full(B, N) if count is None else np.asarray(_to_numpy(count), np.int64)
    page_size = kc.shape[1]
    for b in range(B):
        for n in range(int(count[b])):
            pos = int(start[b]) + n
            pg, slot = table[b, pos // page_size], pos % page_size
            if sc is None:
                kc[pg, slot], vc[pg, slot] = k[b, n], v[b, n]
            else:
                kc[pg, slot], sc[pg, :, 0, slot] = quantise_rows(k[b, n])
                vc[pg, slot], sc[pg, :, 1, slot] = quantise_rows(v[b, n])
    return kc, vc, sc


def cache_read(cache, block_table, seqlens, length: int):
    """[B, length, Hkv, d] float64: the first ``length`` positions of every sequence, zeros past its end."""
    cache = _f64(_to_numpy(cache))
    table = np.asarray(_to_numpy(block_table), np.int64)
    out = np.zeros((table.shape[0], length) + cache.shape[2:])
    for b, n in enumerate(np.asarray(_to_numpy(seqlens), np.int64)):
        n = min(int(n), length)
        out[b, :n] = paged_rows(cache, table[b], n)
    return out


def decode_window(Q, K_cache, V_cache, block_table, seqlens, scale: float, window_left=None):
    """One decode step in which the query, the sequence's last position, sees itself and the ``window_left``
    positions before it (None: all): the plain definition on the visible rows.  Returns O, LSE in float64."""
    Q = _f64(_to_numpy(Q))
    table = np.asarray(_to_numpy(block_table), np.int64)
    nb, nh, d = Q.shape
    K_cache, V_cache = _f64(_to_numpy(K_cache)), _f64(_to_numpy(V_cache))
    hkv, page_size = K_cache.shape[2], K_cache.shape[1]
    O, LSE = np.zeros((nb, nh, d)), np.full((nb, nh), -np.inf)
    for b, n in enumerate(np.asarray(_to_numpy(seqlens), np.int64)):
        n = int(n)
        lo = 0 if window_left is None else max(0, n - 1 - window_left)
        if n == 0:
            continue
        at = np.arange(lo, n)
        k = K_cache[table[b, at // page_size], at % page_size]
        v = V_cache[table[b, at // page_size], at % page_size]
        for h in range(nh):
            g = kv_head(h, nh, hkv)
            o, lse = forward_rows_head(Q[b, h][None, :], k[:, g], v[:, g], [0], scale, False)
            O[b, h], LSE[b, h] = o[0], lse[0]
    return O, LSE
