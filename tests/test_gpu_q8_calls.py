"""Calls of the page plan and the 8-bit cache that a program makes and single calls do not show:
from several host threads at once, and with strides that mean nothing."""
import threading

import numpy as np
import pytest
import torch

from test_gpu_q8 import DEV, _check_plan, _dev, _plan_case

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def ssa():
    import block_sparse_top_summary_b200 as m
    m.load_library()
    return m


def _plans(ssa, batch, stream):
    """One-token plans of ``batch`` rows (24 bytes of shared memory a row)."""
    have = _dev(np.arange(batch) % 40)
    table = torch.arange(batch * 4, dtype=torch.int32, device=DEV).view(batch, 4)
    ring, pool = _dev(np.arange(batch) + 4 * batch), _dev(np.array([0, batch]))
    out = [torch.empty(x, dtype=torch.int32, device=DEV) for x in (batch, batch + 1, batch, 2)]
    return table, *ssa.ssa_page_plan(have, have + 1, table, ring, pool, 16, batch, got=out[0],
                                     cu=out[1], slots=out[2], pool_out=out[3],
                                     stream=stream), have, ring, pool


def _appends(ssa, B, stream):
    """Whole blocks of B rows (576 bytes of shared memory a row in bf16)."""
    d, n = 128, 4
    K, V = (torch.zeros(n, 1, B, d, dtype=torch.int8, device=DEV) for _ in range(2))
    Ks, Vs = (torch.zeros(n, 1, device=DEV) for _ in range(2))
    S = torch.zeros(n, 1, 1, d, device=DEV)
    k = torch.randn(n * B, 1, d, device=DEV).bfloat16()
    new = _dev(np.arange(n * B)), _dev(np.arange(n + 1) * B), _dev(np.full(n, B)), k
    ssa.ssa_append_paged_q8(K, Ks, V, Vs, S, *new, k, B, stream=stream)
    return K, Ks, V, Vs, S, *new


def _decodes(ssa, max_blocks, stream):
    """Routed rows under a table of ``max_blocks`` (4 bytes of shared memory a block)."""
    B, d = 16, 64
    g = torch.Generator().manual_seed(max_blocks)
    K, V = (torch.randint(-127, 128, (50, 1, B, d), generator=g).to(DEV, torch.int8)
            for _ in range(2))
    Ks, Vs = (torch.full((50, 1), 2.0 ** -6, device=DEV) for _ in range(2))
    S = torch.randn(1, 1, max_blocks, d, generator=g).to(DEV)
    table = torch.randint(0, 50, (1, max_blocks), generator=g).to(DEV, torch.int32)
    q, lens = torch.randn(1, 4, d, generator=g).to(DEV), _dev(np.array([16 * 600]))
    ws = torch.empty(ssa.ssa_decode_paged_q8_workspace_size(1, 4, 1, d, B, 8, max_blocks),
                     dtype=torch.uint8, device=DEV)
    O, idx = torch.empty_like(q), torch.empty(1, 1, 10, dtype=torch.int32, device=DEV)
    ssa.ssa_decode_paged_q8(q, K, Ks, V, Vs, S, table, lens, B, 8, O=O, idx=idx, workspace=ws,
                            stream=stream)
    return O, idx, K, V, Ks, Vs, S, table, q, lens, ws


class _Recorder:
    """The library, with the packed arguments of each call kept."""
    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        fn = getattr(self.lib, name)
        if not name.endswith("_words"):
            return fn

        def call(words):
            self.calls.append((fn, words))
            return fn(words)
        return call


@pytest.mark.parametrize("make,sizes", [(_plans, (2100, 8192, 4000)), (_appends, (96, 128, 112)),
                                        (_decodes, (11500, 16384, 13000))])
def test_host_threads_with_calls_of_other_sizes(ssa, monkeypatch, make, sizes):
    # each thread's calls need another amount of shared memory of one kernel; the calls can be
    # repeated on their buffers, and are made without the binding's own work between them
    rec = _Recorder(ssa.load_library())
    monkeypatch.setattr("block_sparse_top_summary_b200.abi.load_library", lambda: rec)
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    tensors = []
    for x, s in zip(sizes, streams):
        with torch.cuda.stream(s):  # (so that the inputs are ready when the call runs)
            tensors.append(make(ssa, x, s))
    torch.cuda.synchronize()
    want = [[t.clone() for t in ts] for ts in tensors]
    start, bad = threading.Barrier(len(sizes)), []

    def work(fn, words):
        start.wait()
        bad.extend(st for st in (fn(words) for _ in range(20000)) if st != 0)

    threads = [threading.Thread(target=work, args=c) for c in rec.calls]
    assert len(threads) == len(sizes)
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert bad == []
    assert all(torch.equal(a, b) for ts, ref in zip(tensors, want) for a, b in zip(ts, ref))


@pytest.mark.parametrize("T,Hkv", [(1, 2), (21, 1), (1, 1), (0, 2)])
def test_strides_of_dimensions_of_one_do_not_matter(ssa, T, Hkv):
    # one token, or one head: k_new and v_new address the same memory whatever that stride is
    B, d = 16, 64
    slots, cu, lens = _dev(np.arange(T)), _dev(np.array([0, T])), _dev(np.array([T]))
    k = torch.randn(T, Hkv, d, device=DEV)
    wide = torch.randn(T, 3 * Hkv, d, device=DEV)
    odd = torch.empty_strided((T, Hkv, d), (Hkv * d if T > 1 else 3, d if Hkv > 1 else 7, 1),
                              device=DEV).copy_(k)

    def run(k, v):
        K, V = (torch.zeros(3, Hkv, B, d, dtype=torch.int8, device=DEV) for _ in range(2))
        Ks, Vs = (torch.zeros(3, Hkv, device=DEV) for _ in range(2))
        S = torch.zeros(1, Hkv, 3, d, device=DEV)
        return ssa.ssa_append_paged_q8(K, Ks, V, Vs, S, slots, cu, lens, k, v, B)

    same = run(k, k)
    got = [run(odd, k), run(k, odd), run(odd, odd)]
    v = wide[:, Hkv:2 * Hkv] if T <= 1 else None  # a slice of a wider row, of one token
    if v is not None:
        for a, b in zip(run(k, v.contiguous()), run(k, v)):
            assert torch.equal(a, b)
    for out in got:
        for a, b in zip(same, out):
            assert torch.equal(a, b)
    if T > 1:  # a stride that does matter still has to agree
        with pytest.raises(ValueError):
            run(k, wide[:, :1])


def test_slices_of_all_heads_past_31_bits(ssa):
    # 16400 heads of 2^21 keys: a sequence's 16-key slices, counted over its heads, pass 2^31.  All
    # blocks are page 0, so a head's result is the attention over its 128 rows there.
    B, d, Hkv, mb = 128, 64, 16400, 16384
    g = torch.Generator(device=DEV).manual_seed(3)
    K, V = (torch.randint(-127, 128, (1, Hkv, B, d), generator=g, device=DEV, dtype=torch.int8)
            for _ in range(2))
    Ks, Vs = (torch.full((1, Hkv), 2.0 ** -6, device=DEV) for _ in range(2))
    q = torch.randn(1, Hkv, d, generator=g, device=DEV)
    table = torch.zeros(1, mb, dtype=torch.int32, device=DEV)
    out, _ = ssa.ssa_decode_paged_q8(q, K, Ks, V, Vs, None, table, _dev(np.array([mb * B])), B,
                                     1 << 20, want_idx=False)
    k, v = (x[0].double() * 2.0 ** -6 for x in (K, V))
    x = (k @ q[0].double()[:, :, None])[..., 0] / 8
    p = torch.softmax(x, -1)
    ref = (p[:, None] @ v)[:, 0]
    mag = (p[:, None] @ v.abs())[:, 0]
    # as in test_gpu_q8_numerics: a logit is off by e, the sums by 2^-17 of the magnitudes;
    # 1.2 M slices a warp make 2^15.2 sums of 32 slices, 2^13 a pair: 2^-24 of the growing sum each
    e = (k.abs() @ q[0].double().abs()[:, :, None]).amax((1, 2)) / 8 * (d / 16 + 4) * 2.0 ** -23
    tol = mag * (2 * e[:, None] + 2.0 ** -17 + 2.0 ** (13 - 24 - 1))
    assert ((out[0].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("n", [4096, 4097, 8192])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_of_many_rows_and_few_tokens(ssa, n, in_place):
    # on both sides of the rows that one block takes: no slot at all, some, and all that are asked
    # for; most rows give pages back or are refused
    for max_new in (0, 1, 300, 8192):
        _check_plan(ssa, _plan_case(n, 16, 9, seed=n + max_new, prompt=5), 16, max_new, in_place)


def test_long_rows_on_two_streams_and_in_one_graph(ssa):
    # runs that are summed in tensor memory (over 32 slices a warp), two calls at once
    B, d, mb = 128, 64, 8192
    g = torch.Generator().manual_seed(5)
    K, V = (torch.randint(-127, 128, (20, 1, B, d), generator=g).to(DEV, torch.int8)
            for _ in range(2))
    Ks, Vs = (torch.full((20, 1), 2.0 ** -6, device=DEV) for _ in range(2))
    table = torch.randint(0, 20, (1, mb), generator=g).to(DEV, torch.int32)
    lens = _dev(np.array([mb * B - 77]))
    qs = [torch.randn(1, 4, d, generator=g).to(DEV) for _ in range(2)]

    def call(q, **kw):
        return ssa.ssa_decode_paged_q8(q, K, Ks, V, Vs, None, table, lens, B, 1 << 20,
                                       want_idx=False, **kw)[0]

    want = [call(q).clone() for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]

    def both():
        out = []
        for q, s in zip(qs, streams):
            s.wait_stream(torch.cuda.current_stream())
            out.append(call(q, stream=s))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        return out

    for _ in range(20):
        for a, b in zip(both(), want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for _ in range(3):
        for a in out:
            a.zero_()
        graph.replay()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
