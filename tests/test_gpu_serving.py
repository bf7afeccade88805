"""The operators around the attention run together, as a serving loop runs them.

A batch of prompts of different lengths goes through norm and rotation, the
causal forward and into the cache; then tokens are decoded one by one, each
through norm and rotation, an append and the paged decode, the step captured
once as a CUDA graph and replayed.
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import exact_io_aware_51_b200 as fa
import oracle
from oracle import serving as S
from tests.helpers import TOL_BF16_REL, TOL_LSE, need_gpu, rel_err
from tests.test_gpu_decode_fp8 import _check as check_decode

B, H, HKV, D, PAGE, MAX_PAGES, ROOM = 3, 8, 2, 128, 16, 20, 320
PROMPTS = [130, 1, 77]


def _projection(N, seed):
    """A packed projection [B, N, H + 2 Hkv, d] as a model hands it over."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, N, H + 2 * HKV, D), generator=g).to(torch.bfloat16).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [True, False])
def test_prompt_then_captured_decode_steps(fp8):
    need_gpu()
    g = torch.Generator().manual_seed(1)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    cos, sin = fa.rope_tables(ROOM, D)
    pages = B * MAX_PAGES
    table = torch.randperm(pages, generator=g).to(torch.int32).view(B, MAX_PAGES).cuda()
    if fp8:
        kc, vc = (torch.zeros((pages, PAGE, HKV, D), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
        sc = torch.zeros((pages, HKV, 2, PAGE), dtype=torch.uint8, device="cuda")
    else:
        kc, vc = (torch.zeros((pages, PAGE, HKV, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        sc = None

    # the prompts, padded to the longest
    N = max(PROMPTS)
    lens = torch.tensor(PROMPTS, dtype=torch.int32, device="cuda")
    at = torch.arange(N, dtype=torch.int32, device="cuda")[None]
    pos = torch.where(at < lens[:, None], at, -1).to(torch.int32)
    x = _projection(N, 2)
    q, k, v = x.split((H, HKV, HKV), dim=2)
    qr, kr = fa.qk_norm_rope(q, k, cos, sin, wq, wk, pos)
    o, _ = fa.fwd(qr, kr, v.contiguous(), causal=True)
    fa.cache_append(kr, v, kc, vc, table, torch.zeros_like(lens), kv_scale=sc, count=lens)
    # the prompt's rows against the oracle (rows behind a prompt's end are not looked at)
    scale = float(np.float32(1 / math.sqrt(D)))
    ro, _ = oracle.forward(qr.float().cpu(), kr.float().cpu(), v.float().cpu(), scale, True)
    for b, n in enumerate(PROMPTS):
        assert rel_err(o[b, :n].cpu(), ro[b, :n]) <= TOL_BF16_REL

    # one decode step on buffers of its own, captured once
    step_x = _projection(1, 3)
    start = lens.clone()

    def step():
        q, k, v = step_x.split((H, HKV, HKV), dim=2)
        qr, kr = fa.qk_norm_rope(q, k, cos, sin, wq, wk, start.view(B, 1))
        fa.cache_append(kr, v, kc, vc, table, start, kv_scale=sc)
        start.add_(1)
        q1 = qr.view(B, H, D)
        if fp8:
            return (qr, kr) + tuple(fa.decode_paged_fp8(q1, kc, vc, sc, table, start))
        return (qr, kr) + tuple(fa.decode_paged(q1, kc, vc, table, start))

    before = [kc.clone(), vc.clone(), None if sc is None else sc.clone()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    kc.copy_(before[0]), vc.copy_(before[1]), start.copy_(lens)
    if sc is not None:
        sc.copy_(before[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr1, kr1, o1, lse1 = step()
    start.copy_(lens)

    ref_k, ref_v = (t.cpu().view(torch.uint8).numpy() if fp8 else t.double().cpu().numpy() for t in (kc, vc))
    ref_s = None if sc is None else sc.cpu().numpy()
    for t in range(5):
        step_x.copy_(_projection(1, 10 + t))
        graph.replay()
        n = lens.cpu() + t
        ref_k, ref_v, ref_s = S.cache_append(kr1.double().cpu(), step_x[:, :, H + HKV:].double().cpu(), ref_k, ref_v,
                                             table.cpu(), n, ref_s)
        got_k = kc.cpu().view(torch.uint8).numpy() if fp8 else kc.double().cpu().numpy()
        assert np.array_equal(got_k, ref_k)
        if fp8:
            assert np.array_equal(sc.cpu().numpy(), ref_s)
            check_decode((qr1.view(B, H, D).cpu(), torch.from_numpy(ref_k), torch.from_numpy(ref_v),
                          torch.from_numpy(ref_s), table.cpu(), n + 1), o1, lse1, 1 / math.sqrt(D))
        else:
            ro, rl = oracle.decode_paged(qr1.view(B, H, D).float().cpu(), ref_k, ref_v, table.cpu(), n + 1, scale)
            assert rel_err(o1.cpu(), ro) <= TOL_BF16_REL
            assert np.max(np.abs(lse1.cpu().numpy() - rl)) <= TOL_LSE
    assert fa.last_device_status()[0] == 0

    # the next part of a prompt reads the cache back
    k2, v2 = fa.cache_read(kc, vc, table, start, ROOM, kv_scale=sc)
    K, V = S.dequantise_cache(ref_k, ref_v, ref_s) if fp8 else (ref_k, ref_v)
    assert torch.equal(k2.cpu(), torch.from_numpy(S.cache_read(K, table.cpu(), start.cpu(), ROOM)).to(torch.bfloat16))
    assert torch.equal(v2.cpu(), torch.from_numpy(S.cache_read(V, table.cpu(), start.cpu(), ROOM)).to(torch.bfloat16))


@pytest.mark.gpu
def test_autograd_sees_what_the_calls_write():
    """A graph that saved a buffer for its backward refuses to run once a call has written it; a buffer that is part
    of a graph itself is refused; an inference tensor is written as any other."""
    need_gpu()
    bf = {"dtype": torch.bfloat16, "device": "cuda"}
    cos, sin = fa.rope_tables(8, 64)
    q, k = torch.randn(2, 3, 4, 64, **bf), torch.randn(2, 3, 2, 64, **bf)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    lens = torch.full((2,), 3, dtype=torch.int32, device="cuda")
    zero = torch.zeros_like(lens)

    def pools(dtype):
        c = [torch.zeros(4, 8, 2, 64, dtype=dtype, device="cuda") for _ in range(2)]
        return c if dtype == torch.bfloat16 else [*c, torch.full((4, 2, 2, 8), 127, dtype=torch.uint8, device="cuda")]

    kv, kv8 = pools(torch.bfloat16), pools(torch.uint8)
    calls = [  # the buffers written, the call
        ([torch.empty_like(q), torch.empty_like(k)],
         lambda b: fa.qk_norm_rope_fwd(q, k, cos, sin, q_out=b[0], k_out=b[1])),
        (pools(torch.bfloat16), lambda b: fa.cache_append(k, k, b[0], b[1], table, zero)),
        (pools(torch.uint8), lambda b: fa.cache_append(k, k, b[0], b[1], table, zero, kv_scale=b[2])),
        ([torch.empty_like(k), torch.empty_like(k)],
         lambda b: fa.cache_read(*kv, table, lens, 3, k_out=b[0], v_out=b[1])),
        ([torch.empty(2, 4, 64, **bf), torch.empty(2, 4, device="cuda")],
         lambda b: fa.decode_paged_fp8(q[:, 0].contiguous(), *kv8, table, lens, out=b[0], lse=b[1])),
    ]
    for bufs, call in calls:
        before = [b._version for b in bufs]
        call(bufs)
        assert all(b._version > v for b, v in zip(bufs, before))
        for i, b in enumerate(bufs):
            if not b.is_floating_point():
                continue
            x = torch.ones((), dtype=b.dtype, device="cuda", requires_grad=True)
            y = (b * x).sum()
            call(bufs)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.backward()
            with pytest.raises(ValueError, match="requires? a gradient"):
                call([b.detach().requires_grad_(True) if j == i else other for j, other in enumerate(bufs)])
            with torch.no_grad():
                call([b.detach().requires_grad_(True) if j == i else other for j, other in enumerate(bufs)])
        with torch.inference_mode():
            call([b.clone() for b in bufs])
    ws = torch.empty(fa.lib().fa_qk_norm_rope_workspace_size(64), dtype=torch.uint8, device="cuda")
    w, v = torch.ones(64, device="cuda"), ws._version
    fa.qk_norm_rope_bwd(q, k, cos, sin, q, k, w, w, workspace=ws)
    assert ws._version > v


@pytest.mark.gpu
def test_tensors_without_storage_are_refused():
    """Under vmap and the other transforms of torch.func a tensor is a wrapper: an error, from every call."""
    need_gpu()
    cos, sin = fa.rope_tables(8, 64)
    q, k = torch.randn(5, 2, 3, 4, 64, device="cuda").bfloat16(), torch.randn(5, 2, 3, 2, 64, device="cuda").bfloat16()
    kc = torch.zeros(5, 4, 8, 2, 64, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(4, 2, 2, 8, dtype=torch.uint8, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    vmap = torch.func.vmap
    for call in (lambda: vmap(lambda a, b: fa.qk_norm_rope(a, b, cos, sin))(q, k),
                 lambda: vmap(lambda a, b: fa.qk_norm_rope_bwd(a, b, cos, sin, a, b)[:2])(q, k),
                 lambda: vmap(lambda c: fa.cache_read(c, c, table, lens, 1, kv_scale=sc))(kc),
                 lambda: vmap(lambda a: fa.cache_append(a, a, kc[0], kc[0], table, lens, kv_scale=sc))(k),
                 lambda: vmap(lambda a: fa.decode_paged_fp8(a[:, 0].contiguous(), kc[0], kc[0], sc, table, lens))(q),
                 lambda: torch.func.grad(lambda a: fa.qk_norm_rope(a, k[0], cos, sin)[0].float().sum())(q[0])):
        with pytest.raises(RuntimeError):
            call()
    qo, _ = fa.qk_norm_rope(q[0], k[0], cos, sin)  # the interpreter and the binding are well
    assert torch.isfinite(qo).all() and fa.last_device_status()[0] == 0


@pytest.mark.gpu
def test_two_threads_on_streams_of_their_own():
    """The calls give up the interpreter's lock: two threads run them at once, each on a stream that is not the
    current one, with the results of one thread alone."""
    import threading

    need_gpu()
    cos, sin = fa.rope_tables(4096, D)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    length, steps = 3000, 40

    def run(seed, stream, out):
        try:
            x = _projection(1, seed).expand(B, 1, H + 2 * HKV, D)
            q, k, v = x.split((H, HKV, HKV), dim=2)
            pages = (length + steps + PAGE) // PAGE
            table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
            kc, vc = (torch.full((B * pages, PAGE, HKV, D), 0x38, dtype=torch.uint8, device="cuda") for _ in range(2))
            sc = torch.full((B * pages, HKV, 2, PAGE), 120, dtype=torch.uint8, device="cuda")
            lens = [torch.full((B,), length + t, dtype=torch.int32, device="cuda") for t in range(steps + 1)]
            torch.cuda.current_stream().synchronize()
            got = []
            for t in range(steps):
                qr, kr = fa.qk_norm_rope_fwd(q, k, cos, sin, w, w, lens[t].view(B, 1), stream=stream)
                fa.cache_append(kr, v, kc, vc, table, lens[t], kv_scale=sc, stream=stream)
                got.append((*fa.decode_paged_fp8(qr.view(B, H, D), kc, vc, sc, table, lens[t + 1], stream=stream), kr))
            got.append(fa.cache_read(kc, vc, table, lens[steps], length + steps, kv_scale=sc, stream=stream))
            stream.synchronize()
            out.append([y.cpu() for pair in got for y in pair])
        except BaseException as e:  # noqa: BLE001 - handed to the test
            out.append(e)

    streams = [torch.cuda.Stream() for _ in range(2)]
    want = [[], []]
    for i in range(2):
        run(50 + i, streams[i], want[i])
    got = [[], []]
    threads = [threading.Thread(target=run, args=(50 + i, streams[i], got[i])) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert not isinstance(a[0], BaseException) and not isinstance(b[0], BaseException), (a[0], b[0])
        assert len(a[0]) == len(b[0]) and all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    assert fa.last_device_status()[0] == 0


@pytest.mark.gpu
def test_two_graphs_and_an_eager_call_do_not_share_scratch():
    """Split decodes captured twice, replayed on two streams at once beside an eager one: each has partials of its own."""
    need_gpu()
    from tests.test_gpu_decode_fp8 import _make
    a = [t.cuda() for t in _make(1, 8, 2, 128, 16, [6000], seed=41)]
    b = [t.cuda() for t in _make(1, 8, 2, 128, 16, [5000], seed=42)]
    assert fa.decode_fp8_workspace_size(1, 8, 2, 128, 16, a[4].shape[1]) > 0
    want = [tuple(t.clone() for t in fa.decode_paged_fp8(*x)) for x in (a, b)]
    graphs, outs = [], []
    for x in (a, b):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(fa.decode_paged_fp8(*x))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        eager = fa.decode_paged_fp8(*a, stream=streams[2])
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for got, ref in zip((*outs, eager), (*want, want[0])):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
