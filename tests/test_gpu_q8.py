"""GPU parity of the page plan and of the paged 8-bit cache (append and decode)
with the fp64 oracle.

The plan's outputs are whole numbers and have to be equal.  Codes and scales are
exact too: scales are powers of two, so x / scale is exact and only the rounding
to a code is left, which the definition fixes.  A summary is an fp32 sum of B
codes (whole multiples of one step, below 2^24 of them in the int8 case) times a
factor: at most B roundings of half a step, 2^-24, of the partial sums.

Decode in fp32.  Per logit, with A = max_t scale sum_i |q_i k_ti|: splitting q in two f16
leaves 2^-22, and d / 16 accumulations each at most a step, 2^-23, of a partial
sum no larger than A; with the products by scales below 2^-22.  So
|dx| <= A (d / 16 + 4) 2^-23 =: e.  Probabilities then move by a factor within
exp(2 e), P's split and ex2 by 2^-21, and the sums of at most 2^10 fp32 partial results by
2^-20 of sum p |v| <= Vmax.  |dO| <= Vmax (2 e + 2^-19).  In bf16 P is one f16: half a step of
each p, 2^-11, makes 2^-11 Vmax; and half a step of the result, 2^-8 |O|, comes on top.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
DEV = "cuda"
TORCH = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8, "bf16": torch.bfloat16,
         "f32": torch.float32}


@pytest.fixture(scope="module")
def ssa():
    import block_sparse_top_summary_b200 as m
    m.load_library()
    return m


def _dev(x, t=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(DEV, t)


def _np(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------ plan
def _plan_case(n, B, mb, seed, spare=5, prompt=60):
    r = np.random.default_rng(seed)
    cap = B * mb
    have = r.integers(0, cap + 1, n)
    have[r.random(n) < 0.2] = 0
    have[r.random(n) < 0.2] = cap // 2 // B * B
    kind = r.integers(0, 5, n)
    want = np.where(kind == 0, have, np.where(kind == 1, np.minimum(cap, have + 1), np.where(
        kind == 2, np.minimum(cap, have + r.integers(0, prompt, n)), np.where(
            kind == 3, 0, np.maximum(0, have - r.integers(0, 2 * B, n))))))
    keep = np.where(r.random(n) < 0.3, r.integers(0, mb + 1, n), 0)
    hb = -(-have // B)
    used = int(hb.sum())
    need = int(np.maximum(-(-want // B) - hb, 0).sum())
    pages = used + need + spare
    order = r.permutation(pages)
    table = np.full((n, mb), -7)
    table[np.arange(mb)[None] < hb[:, None]] = order[:used]
    head = int(r.integers(0, pages))
    free = pages - used
    ring = np.full(pages, -9)
    ring[(head + np.arange(free)) % pages] = order[used:]
    return have, want, keep, table, ring, [head, free]


def _check_plan(ssa, case, B, max_new, in_place=False):
    have, want, keep, table, ring, pool = case
    ref = O.page_plan(have, want, keep, table, ring, pool, B, max_new)
    h, tb, rg, pl = _dev(have), _dev(table), _dev(ring), _dev(np.array(pool))
    kw = dict(got=h, pool_out=pl) if in_place else {}
    got, cu, slots, pool_out = ssa.ssa_page_plan(
        h, _dev(want), tb, rg, pl, B, max_new, keep=None if keep is None else _dev(keep), **kw)
    torch.cuda.synchronize()
    for name, a, b in zip(("got", "cu", "slots", "pool", "table", "ring"),
                          (got, cu, slots, pool_out, tb, rg), ref):
        assert np.array_equal(a.cpu().numpy(), b), name
    return ref


@pytest.mark.parametrize("n,B,mb", [(1, 64, 1), (3, 16, 5), (33, 48, 9), (1000, 16, 4),
                                    (1025, 64, 7), (5000, 128, 3), (8192, 16, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_the_oracle(ssa, n, B, mb, in_place):
    for seed in range(3):
        case = _plan_case(n, B, mb, 10 * seed + n)
        total = int(np.maximum(case[1] - case[0], 0).sum())
        _check_plan(ssa, case, B, total + 17, in_place)


@pytest.mark.parametrize("n,B,mb,prompt", [(40, 16, 64, 1000), (700, 48, 20, 90),
                                           (9, 128, 40, 5000), (3000, 32, 3, 30),
                                           (7, 16, 5000, 70000)])
def test_plan_of_many_tokens(ssa, n, B, mb, prompt):
    # more than 8192 slots: a cluster and a kernel for the slots; short and long rows, up to
    # thousands of pages; refused ones
    for seed in range(2):
        have, want, keep, table, ring, (head, count) = _plan_case(n, B, mb, seed + n, prompt=prompt)
        total = int(np.maximum(want - have, 0).sum())
        for free, room in ((count, total + 3), (count, 3 * total // 4), (count // 2, total)):
            _check_plan(ssa, (have, want, keep, table, ring, [head, free]), B, max(room, 8193),
                        in_place=seed == 1)


@pytest.mark.parametrize("max_new", [0, 1, 37, 300])
@pytest.mark.parametrize("free", [0, 1, 9])
def test_plan_refuses_rows_beyond_pages_or_tokens(ssa, max_new, free):
    have, want, keep, table, ring, (head, count) = _plan_case(64, 16, 6, 5)
    case = (have, want, keep, table, ring, [head, min(free, count)])
    ref = _check_plan(ssa, case, 16, max_new)
    assert (ref[0] != want).any()  # some row was refused


def test_plan_lengths_out_of_range_and_sums_past_31_bits(ssa):
    have, want, keep, table, ring, pool = _plan_case(9, 32, 4, 6)
    have[1], want[1] = -1, 5
    have[2], want[2] = 0, 32 * 4 + 1
    have[3], want[3] = 32 * 4 + 1, 3
    want[4] = -3
    have[5], want[5] = 2 ** 31 - 1, -2 ** 31
    _check_plan(ssa, (have, want, keep, table, ring, pool), 32, 500)
    # three rows ask for 10^9 tokens each, a fourth for one
    mb = 8_000_000
    big = np.full((4, mb), -1, np.int32)
    have, want = np.zeros(4, np.int64), np.array([10 ** 9, 10 ** 9, 10 ** 9, 1])
    _check_plan(ssa, (have, want, None, big, np.arange(50), [3, 20]), 128, 1000)
    _check_plan(ssa, (have, want[::-1].copy(), None, big, np.arange(50), [3, 20]), 128, 1000)


def test_tensors_of_another_kind_are_refused(ssa):
    B, d, L = 16, 64, [20]
    cache = _cache("i8", d, B, 2, L, seed=30)
    K, Ks, V, Vs, S = (x.to(DEV) for x in cache[:5])
    table, lens = _dev(cache[5]), _dev(np.asarray(L))
    q = torch.randn(1, 4, d, device=DEV)

    def call(q=q, K=K, Ks=Ks, V=V, S=S, table=table, lens=lens, **kw):
        return ssa.ssa_decode_paged_q8(q, K, Ks, V, Vs, S, table, lens, B, 1 << 20, **kw)

    call()
    for bad in (dict(q=q.cpu()), dict(table=table.cpu()), dict(S=S[:, :1]), dict(lens=lens[:0]),
                dict(K=K.transpose(0, 1)), dict(q=q.transpose(1, 2)), dict(Ks=Ks[:, :1])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q=q.half()), dict(table=table.long()), dict(V=V.view(torch.uint8)),
                dict(K=K.view(torch.uint8)), dict(Ks=Ks.double()), dict(O=torch.empty_like(q).bfloat16())):
        with pytest.raises(TypeError):
            call(**bad)
    wide = torch.zeros(1, 9, dtype=torch.int32, device=DEV)
    with pytest.raises(ssa.SSAError):  # too small a workspace
        ssa.ssa_decode_paged_q8(q, K, Ks, V, Vs, torch.zeros(1, 2, 9, d, device=DEV), wide, lens, B,
                                2, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ssa.SSAError):  # no summaries, and blocks to choose from
        ssa.ssa_decode_paged_q8(q, K, Ks, V, Vs, None, wide, lens, B, 2)
    with pytest.raises(TypeError):
        ssa.ssa_page_plan(lens.long(), lens, table, lens, lens, B, 4)
    torch.cuda.synchronize()


def test_plan_bad_pool_state_stays_in_bounds(ssa):
    # a head or a count outside the ring: clamped; a page that comes back when
    # the ring is full: dropped
    have, want = np.array([40, 16, 0]), np.array([0, 17, 20])
    table = np.array([[0, 1, 2], [3, -1, -1], [-1, -1, -1]])
    for pool, seen in (([-5, 99], [0, 4]), ([7, -2], [3, 0])):
        h, tb, rg, pl = _dev(have), _dev(table), _dev(np.arange(4)), _dev(np.array(pool))
        got, cu, slots, out = ssa.ssa_page_plan(h, _dev(want), tb, rg, pl, 16, 64)
        torch.cuda.synchronize()
        ref = O.page_plan(have, want, None, table, np.arange(4), seen, 16, 64)
        for a, b in zip((got, cu, slots, out, tb, rg), ref):
            assert np.array_equal(a.cpu().numpy(), b)


def test_plan_undone_and_repeated_keeps_every_page_once(ssa):
    # 40 steps of growth and shrinkage: table and ring together hold each page once
    r = np.random.default_rng(7)
    n, B, mb, pages = 50, 16, 8, 260
    have = torch.zeros(n, dtype=torch.int32, device=DEV)
    table = torch.full((n, mb), -1, dtype=torch.int32, device=DEV)
    ring = torch.arange(pages, dtype=torch.int32, device=DEV)
    pool = _dev(np.array([0, pages]))
    for _ in range(40):
        h = have.cpu().numpy()
        want = np.clip(h + r.integers(-60, 61, n), 0, B * mb)
        ssa.ssa_page_plan(have, _dev(want), table, ring, pool, B, 4096, got=have, pool_out=pool)
        h, tb, rg = have.cpu().numpy(), table.cpu().numpy(), ring.cpu().numpy()
        head, count = pool.tolist()
        held = [int(p) for b in range(n) for p in tb[b, : -(-h[b] // B)]]
        free = [int(rg[(head + i) % pages]) for i in range(count)]
        assert sorted(held + free) == list(range(pages))


# ---------------------------------------------------------------------- append
def _append_case(fmt, dtype, d, B, Hkv, have, new, seed, refuse=()):
    """A cache with some tokens in it and the new tokens of a ragged batch."""
    r = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    n = len(have)
    have, new = np.asarray(have), np.asarray(new)
    L = have + new
    nb = -(-L // B)
    mb = max(1, int(nb.max()))
    pages = int(nb.sum()) + 3
    order = r.permutation(pages)
    first = np.concatenate([[0], np.cumsum(nb)])
    cu = np.concatenate([[0], np.cumsum(new)])
    slots = np.concatenate([order[first[b] + np.arange(have[b], L[b]) // B] * B
                            + np.arange(have[b], L[b]) % B for b in range(n)] + [[-1, -1, -1]])
    seqlens = L.copy()
    for b in refuse:
        slots[cu[b]:cu[b + 1]] = -1
        seqlens[b] = have[b]
    if fmt == "i8":
        K, V = (torch.randint(-127, 128, (pages, Hkv, B, d), generator=g).to(torch.int8)
                for _ in range(2))
    else:
        K, V = ((100 * torch.randn(pages, Hkv, B, d, generator=g)).clamp(-448, 448)
                .to(torch.float8_e4m3fn) for _ in range(2))
    Ks, Vs = (torch.exp2(torch.randint(-9, -3, (pages, Hkv), generator=g).float())
              for _ in range(2))
    T = len(slots)
    x = [torch.randn(T, Hkv, d, generator=g)
         * torch.exp2(torch.randint(-4, 3, (T, Hkv, 1), generator=g).float()) for _ in range(2)]
    return dict(K=K, Ks=Ks, V=V, Vs=Vs, S=torch.randn(n, Hkv, mb, d, generator=g),
                slots=slots, cu=cu, seqlens=seqlens, k=x[0].to(TORCH[dtype]),
                v=x[1].to(TORCH[dtype]), B=B, fmt=fmt)


def _run_append(ssa, c, k=None, v=None, S=True, stream=None):
    out = [c[n].to(DEV) for n in ("K", "Ks", "V", "Vs")]
    s = c["S"].to(DEV) if S else None
    ssa.ssa_append_paged_q8(*out, s, _dev(c["slots"]), _dev(c["cu"]), _dev(c["seqlens"]),
                            c["k"].to(DEV) if k is None else k, c["v"].to(DEV) if v is None else v,
                            c["B"], max_blocks=c["S"].shape[2])
    torch.cuda.synchronize()
    return (*out, s)


def _check_append(c, got, S=True):
    ref = O.append_paged_q8(_np(c["K"]), _np(c["Ks"]), _np(c["V"]), _np(c["Vs"]), _np(c["S"]),
                            c["slots"], c["cu"], c["seqlens"], _np(c["k"]), _np(c["v"]), c["B"],
                            c["fmt"])
    for name, a, b in zip(("K", "Ks", "V", "Vs"), got, ref):
        assert np.array_equal(_np(a), b, equal_nan=True), name
    if S:
        a, b = _np(got[4]), ref[4]
        changed = b != _np(c["S"])
        assert np.array_equal(a[~changed], b[~changed], equal_nan=True)
        big = O.QMAX[c["fmt"]] * np.nanmax(ref[1])  # no value is larger
        # S is fp32: 3.4028234e38 is held as the e4m3 code 256 times 2^120 = 2^128, whose
        # mean no fp32 number below infinity is nearest to
        with np.errstate(over="ignore"):
            b32 = b.astype(np.float32)
        fine = np.isfinite(b32)
        assert np.array_equal(a[~fine], b32[~fine], equal_nan=True)
        assert np.all(np.abs(a - b)[fine] <= (c["B"] + 2) * 2.0 ** -24 * big)
    return ref


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype,d,B,Hkv", [("bf16", 128, 64, 2), ("f32", 64, 16, 3),
                                           ("bf16", 64, 48, 1), ("f32", 128, 128, 2),
                                           ("bf16", 128, 128, 5)])
def test_append_matches_the_oracle(ssa, fmt, dtype, d, B, Hkv):
    # empty rows, a first token, ends on and around a block's end, several blocks
    have = [0, 0, B - 1, B - 1, 3, 0, 2 * B, 5, B // 2, 0]
    new = [1, 0, 1, 2, B - 3, 3 * B, 7, 2 * B + 3, B // 2, B]
    c = _append_case(fmt, dtype, d, B, Hkv, have, new, seed=d + B, refuse=(6,))
    _check_append(c, _run_append(ssa, c))


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_append_token_by_token_grows_the_scale(ssa, fmt):
    # one sequence, rows whose size grows by 2^(1/4) a token: the scale grows many times
    B, d, Hkv = 16, 64, 2
    c = _append_case(fmt, "f32", d, B, Hkv, [0], [2 * B], seed=3)
    c["k"] *= torch.exp2(torch.arange(len(c["k"])) / 4)[:, None, None]
    state = [c[n].to(DEV) for n in ("K", "Ks", "V", "Vs")] + [c["S"].to(DEV)]
    ref = [_np(x) for x in state]
    for i in range(2 * B):
        slots, cu, L = c["slots"][i:i + 1], np.array([0, 1]), np.array([i + 1])
        ssa.ssa_append_paged_q8(*state, _dev(slots), _dev(cu), _dev(L),
                                c["k"][i:i + 1].to(DEV), c["v"][i:i + 1].to(DEV), B)
        ref = O.append_paged_q8(*ref, slots, cu, L, _np(c["k"][i:i + 1]), _np(c["v"][i:i + 1]), B,
                                fmt)
        for a, b in zip(state[:4], ref):
            assert np.array_equal(_np(a), b)
    big = O.QMAX[fmt] * ref[1].max()
    assert np.abs(_np(state[4]) - ref[4]).max() <= (B + 2) * 2.0 ** -24 * big


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_append_odd_values(ssa, fmt):
    # zeros, subnormals, the largest fp32, ties, a NaN and infinities: the block of
    # these alone gets a NaN scale, and row 0 of the next turn clears it
    B, d, Hkv = 16, 64, 1
    have, new = [0, 0, 0, 0, 4, 0, 0], [B, B, B, 5, 3, B + 1, 7]
    c = _append_case(fmt, "f32", d, B, Hkv, have, new, seed=11)
    k, cu = c["k"], c["cu"]
    k[cu[0]:cu[1]] = 0
    k[cu[1]:cu[2]] *= 2.0 ** -140
    k[cu[2]:cu[3]] = 3.4028234e38 * (torch.arange(d) - 31).sign()
    k[cu[3]:cu[4]] = torch.arange(5 * d).view(5, 1, d) / 2 - 63.5 if fmt == "i8" else k[cu[3]:cu[4]]
    k[cu[4] + 1, 0, 5] = float("nan")
    k[cu[5] + B, 0, 0] = float("inf")
    c["v"][cu[6] + 2, 0, 1] = float("-inf")
    ref = _check_append(c, _run_append(ssa, c))
    assert np.isnan(ref[1]).sum() == 2 and np.isnan(ref[3]).sum() == 1
    # a block with a NaN scale keeps it while tokens are added to it ...
    at = int(c["slots"][cu[4]]) // B
    c2 = dict(c, K=torch.from_numpy(ref[0]).to(TORCH[fmt]), Ks=torch.from_numpy(ref[1]).float(),
              V=torch.from_numpy(ref[2]).to(TORCH[fmt]), Vs=torch.from_numpy(ref[3]).float(),
              slots=np.array([at * B + 7, at * B]), cu=np.array([0, 1, 2]),
              seqlens=np.array([8, 1]), k=torch.ones(2, 1, d), v=torch.ones(2, 1, d),
              S=torch.zeros(2, 1, 1, d))
    only = {**c2, "slots": c2["slots"][:1], "cu": c2["cu"][:2], "seqlens": c2["seqlens"][:1],
            "k": c2["k"][:1], "v": c2["v"][:1], "S": c2["S"][:1]}
    assert np.isnan(_check_append(only, _run_append(ssa, only))[1][at, 0])
    # ... and loses it when the page is begun again
    again = {**c2, "slots": c2["slots"][1:], "cu": c2["cu"][:2], "seqlens": c2["seqlens"][1:],
             "k": c2["k"][1:], "v": c2["v"][1:], "S": c2["S"][1:]}
    assert np.isfinite(_check_append(again, _run_append(ssa, again))[1][at, 0])


def test_append_strided_rows_and_no_summaries(ssa):
    # the K of a one-sequence prefill, [1, Hkv, N, d], and rows of a wider tensor
    B, d, Hkv = 64, 128, 3
    c = _append_case("e4m3", "bf16", d, B, Hkv, [10], [150], seed=12)
    ref = _run_append(ssa, c)
    T = len(c["slots"])
    kb = c["k"].transpose(0, 1).contiguous().to(DEV)[None]
    vb = c["v"].transpose(0, 1).contiguous().to(DEV)[None]
    got = _run_append(ssa, c, k=kb[0].transpose(0, 1), v=vb[0].transpose(0, 1))
    wide = torch.zeros(T, 2, Hkv + 1, d, dtype=torch.bfloat16, device=DEV)
    wide[:, 0, :Hkv] = c["k"].to(DEV)
    wide[:, 1, :Hkv] = c["v"].to(DEV)
    got2 = _run_append(ssa, c, k=wide[:, 0, :Hkv], v=wide[:, 1, :Hkv], S=False)
    for a, b, e in zip(ref[:4], got, got2):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(a.view(torch.uint8), e.view(torch.uint8))
    assert torch.equal(ref[4], got[4])
    with pytest.raises(ValueError):
        _run_append(ssa, c, k=wide[:, 0, :Hkv], v=c["v"].to(DEV))
    with pytest.raises(ssa.SSAError):  # rows that do not begin on 16 bytes
        odd = torch.zeros(T, Hkv, d + 2, dtype=torch.bfloat16, device=DEV)[:, :, :d]
        _run_append(ssa, c, k=odd, v=odd)


def test_append_slots_that_are_not_the_blocks_are_left_out(ssa):
    B, d = 32, 64
    c = _append_case("i8", "bf16", d, B, 2, [0, 40, 7], [5, 3, 4], seed=13)
    c["slots"][0] += 1                       # not the place of position 0
    c["slots"][5:8] += len(c["K"]) * B       # beyond the pool
    before = [c[n].clone() for n in ("K", "Ks", "V", "Vs")]
    got = _run_append(ssa, c)
    third = int(c["slots"][8]) // B
    for a, b in zip(got[:4], before):
        keep = [p for p in range(len(b)) if p != third]
        assert torch.equal(a.cpu()[keep], b[keep])
    c["slots"][:8] = -1
    c["seqlens"][:2] = [0, 40]
    _check_append(c, got)


# ---------------------------------------------------------------------- decode
def _cache(fmt, d, B, Hkv, L, seed, poison=True, loud=1.0):
    """Codes, scales, page table (shuffled) and summaries of sequences of lengths L."""
    r = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    n = len(L)
    nb = [-(-max(x, 0) // B) for x in L]
    mb = max(max(nb), 1)
    pages = sum(nb) + 4
    order = r.permutation(pages)
    table = np.full((n, mb), -1)
    at = 0
    K, V = (torch.randn(pages, Hkv, B, d, generator=g) * loud for _ in range(2))
    out = []
    for x in (K, V):
        s = torch.from_numpy(np.array([[O.q8_scale(float(x[p, h].abs().max()), fmt)
                                        for h in range(Hkv)] for p in range(pages)]))
        y = x.double() / s[:, :, None, None]
        out += [torch.from_numpy(O.nearest_code(y.numpy(), fmt)).to(TORCH[fmt]), s.float()]
    K, Ks, V, Vs = out
    S = torch.zeros(n, Hkv, mb, d)
    for b in range(n):
        for j in range(nb[b]):
            p = table[b, j] = order[at]
            at += 1
            S[b, :, j] = (K[p].double().mean(dim=1) * Ks[p].double()[:, None]).float()
            rows = L[b] - j * B
            if poison and rows < B:  # rows behind the sequence: NaN codes, or the lowest
                bad = 0x7F if fmt == "e4m3" else -128
                K.view(torch.int8)[p, :, rows:] = bad
                V.view(torch.int8)[p, :, rows:] = bad
    return K, Ks, V, Vs, S, table


def _tolerance(q, K, Ks, Ls, scale, V, Vs, dtype, ref):
    d = q.shape[-1]
    A = scale * np.abs(q).sum(-1).max() * np.abs(O.q8_values(np.nan_to_num(K), Ks)).max()
    # sum |q_i k_i| <= |q| |k| (Cauchy), far below the product of the extremes
    A = min(A, scale * np.linalg.norm(q, axis=-1).max()
            * np.linalg.norm(O.q8_values(np.nan_to_num(K), Ks), axis=-1).max())
    e = A * (d / 16 + 4) * 2.0 ** -23
    vmax = np.abs(O.q8_values(np.nan_to_num(V), Vs)).max()
    tol = vmax * (2 * e + 2.0 ** -19)
    return tol + (2.0 ** -11 * vmax + 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0)


def _run_decode(ssa, cache, q, L, B, topk, S=True, **kw):
    K, Ks, V, Vs, Sm, table = cache
    args = [x.to(DEV) for x in (K, Ks, V, Vs)]
    out = ssa.ssa_decode_paged_q8(q.to(DEV), *args, Sm.to(DEV) if S else None, _dev(table),
                                  _dev(np.asarray(L)), B, topk, **kw)
    torch.cuda.synchronize()
    return out


def _check_decode(cache, q, L, B, topk, got, idx, dtype, scale=None):
    K, Ks, V, Vs, S, table = cache
    L = np.asarray(L)
    mb = table.shape[1]
    ok = (L >= 1) & (L <= mb * B)
    qn = _np(q)
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    ref, _, oi, _ = O.decode_paged_q8(qn[ok], _np(K), _np(Ks), _np(V), _np(Vs), table[ok], L[ok],
                                      B, min(topk, mb), S=_np(S)[ok], scale=scale)
    assert np.array_equal(idx.cpu().numpy()[ok], oi)
    assert (idx.cpu().numpy()[~ok] == -1).all() and (got.cpu()[torch.from_numpy(~ok)] == 0).all()
    err = np.abs(_np(got)[ok] - ref)
    assert np.all(err <= _tolerance(qn, _np(K), _np(Ks), L, scale, _np(V), _np(Vs), dtype, ref)), \
        err.max()


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype,d,B,Hq,Hkv", [("bf16", 128, 64, 8, 2), ("f32", 128, 64, 8, 1),
                                              ("f32", 64, 16, 3, 3), ("bf16", 64, 48, 14, 2),
                                              ("f32", 128, 128, 5, 1), ("bf16", 64, 112, 8, 4)])
@pytest.mark.parametrize("topk", [0, 2, 1 << 30])
def test_decode_matches_the_oracle(ssa, fmt, dtype, d, B, Hq, Hkv, topk):
    L = [9 * B + 5, 1, B, 0, B + 1, 2 * B + 15, 17, -4, 10 * B, 11 * B, 7 * B + B // 2]
    cache = list(_cache(fmt, d, B, Hkv, L, seed=d + B + Hq))
    L[9] += 1  # one more than its pages hold: out of range
    q = torch.randn(len(L), Hq, d, generator=torch.Generator().manual_seed(1)).to(TORCH[dtype])
    got, idx = _run_decode(ssa, cache, q, L, B, topk, S=topk < 9)
    _check_decode(cache, q, L, B, topk, got, idx, dtype)


@pytest.mark.parametrize("fmt,dtype,d", [("e4m3", "bf16", 128), ("i8", "f32", 64)])
@pytest.mark.parametrize("n,L,B,topk", [(1, 20011, 64, 1 << 30), (2, 9000, 16, 7),
                                        (70, 300, 32, 3), (5, 4096, 128, 1 << 30)])
def test_decode_long_rows_and_many_rows(ssa, fmt, dtype, d, n, L, B, topk):
    lens = [max(1, L - 37 * b) for b in range(n)]
    cache = _cache(fmt, d, B, 1, lens, seed=n)
    q = torch.randn(n, 4, d, generator=torch.Generator().manual_seed(2)).to(TORCH[dtype])
    got, idx = _run_decode(ssa, cache, q, lens, B, topk)
    _check_decode(cache, q, lens, B, topk, got, idx, dtype)


@pytest.mark.parametrize("topk", [1, 31, 200, 256, 257, 900])
@pytest.mark.parametrize("ties", [False, True])
def test_decode_selection_of_long_rows(ssa, topk, ties):
    # up to 1100 candidates; with ties, few distinct scores: lists longer than the
    # quick selection holds, and equal scores go to the lower block
    B, d, L = 16, 64, [16 * 1102, 16 * 260 + 3, 16 * 1000]
    cache = list(_cache("i8", d, B, 2, L, seed=20))
    q = torch.randn(3, 4, d, generator=torch.Generator().manual_seed(21))
    if ties:
        few = torch.randn(3, 2, 5, d, generator=torch.Generator().manual_seed(22))
        which = torch.randint(0, 5, cache[4].shape[:3], generator=torch.Generator().manual_seed(23))
        cache[4] = torch.gather(few, 2, which[..., None].expand(*which.shape, d)).contiguous()
    got, idx = _run_decode(ssa, cache, q, L, B, topk)
    _check_decode(cache, q, L, B, topk, got, idx, "f32")


def test_decode_selection_at_the_largest_cache(ssa):
    # 16384 blocks, the most that a cache may have
    B, d, L = 16, 64, [16 * 16384 - 3, 16 * 9000]
    cache = list(_cache("e4m3", d, B, 1, L, seed=24))
    q = torch.randn(2, 8, d, generator=torch.Generator().manual_seed(25))
    for topk in (32, 100):
        got, idx = _run_decode(ssa, cache, q, L, B, topk)
        _check_decode(cache, q, L, B, topk, got, idx, "f32")


@pytest.mark.parametrize("topk", [1, 1 << 30])
def test_decode_more_rows_than_threads(ssa, topk):
    # over 384 rows the slices' sums come from the route kernel; some rows are empty
    B, d, n = 16, 64, 700
    r = np.random.default_rng(26)
    L = r.integers(0, 90, n)
    cache = _cache("i8", d, B, 1, L.tolist(), seed=26)
    q = torch.randn(n, 2, d, generator=torch.Generator().manual_seed(27)).bfloat16()
    got, idx = _run_decode(ssa, cache, q, L, B, topk)
    _check_decode(cache, q, L, B, topk, got, idx, "bf16")


def test_pools_past_4_gb(ssa):
    # the last pages of pools of 5.2 GB: byte offsets past 32 bits
    B, d, Hkv, pages = 128, 128, 8, 40000
    K = torch.empty(pages, Hkv, B, d, dtype=torch.int8, device=DEV)
    V = torch.empty_like(K)
    Ks, Vs = (torch.zeros(pages, Hkv, device=DEV) for _ in range(2))
    L = np.array([300, 129])
    table = np.array([[pages - 1, 35000, pages - 3], [34000, pages - 2, -1]])
    cu = np.array([0, 300, 429])
    slots = np.concatenate([table[b, np.arange(n) // B] * B + np.arange(n) % B
                            for b, n in enumerate(L)])
    g = torch.Generator().manual_seed(28)
    k, v = (torch.randn(429, Hkv, d, generator=g) for _ in range(2))
    S = torch.zeros(2, Hkv, 3, d, device=DEV)
    ssa.ssa_append_paged_q8(K, Ks, V, Vs, S, _dev(slots), _dev(cu), _dev(L), k.to(DEV), v.to(DEV),
                            B)
    q = torch.randn(2, 16, d, generator=g)
    used = table[table >= 0]
    small = np.full_like(table, -1)
    small[table >= 0] = np.arange(5)
    at = torch.from_numpy(used).to(DEV)
    cache = [x[at].cpu() for x in (K, Ks, V, Vs)] + [S.cpu(), small]
    zero = torch.zeros(5, Hkv, B, d, dtype=torch.int8)
    one = torch.zeros(5, Hkv)
    ref = O.append_paged_q8(_np(zero), _np(one), _np(zero), _np(one), None,
                            np.concatenate([small[b, np.arange(n) // B] * B + np.arange(n) % B
                                            for b, n in enumerate(L)]), cu, L, _np(k), _np(v), B,
                            "i8")
    for b in range(2):  # rows behind a sequence are never written: compare the others
        for p in range(L[b]):
            i, row = small[b, p // B], p % B
            assert np.array_equal(_np(cache[0][i, :, row]), ref[0][i, :, row])
    assert np.array_equal(_np(cache[1]), ref[1]) and np.array_equal(_np(cache[3]), ref[3])
    out, idx = ssa.ssa_decode_paged_q8(q.to(DEV), K, Ks, V, Vs, S, _dev(table), _dev(L), B, 1)
    torch.cuda.synchronize()
    for x in (cache[0], cache[2]):  # not written, and not to matter
        x[2, :, 300 - 256:] = 0
        x[4, :, 1:] = 0
    _check_decode(cache, q, L, B, 1, out, idx, "f32")


def test_decode_nan_query_stays_in_its_head(ssa):
    B, d, L = 16, 64, [200, 90]
    cache = _cache("e4m3", d, B, 2, L, seed=31)
    q = torch.randn(2, 8, d, generator=torch.Generator().manual_seed(31))
    clean, _ = _run_decode(ssa, cache, q, L, B, 1 << 20)
    q[0, 1, 3], q[1, 6, 0] = float("nan"), float("inf")
    got, _ = _run_decode(ssa, cache, q, L, B, 1 << 20)
    bad = torch.zeros(2, 8, dtype=torch.bool)
    bad[0, 1] = bad[1, 6] = True
    assert torch.isnan(got.cpu()[bad]).all()
    assert torch.equal(got.cpu()[~bad], clean.cpu()[~bad])


def test_decode_scale_argument_loud_caches_and_quiet_queries(ssa):
    # scales far from 1 on both sides: codes and f16 parts must not leave their range
    B, d, L = 32, 64, [200, 77]
    q = torch.randn(2, 4, d, generator=torch.Generator().manual_seed(3))
    for loud, quiet in ((2.0 ** 30, 2.0 ** -30), (2.0 ** -30, 2.0 ** 30)):
        cache = _cache("e4m3", d, B, 2, L, seed=4, loud=loud)
        for scale in (0.3, 1e-4):
            got, idx = _run_decode(ssa, cache, q * quiet, L, B, 2, scale=scale)
            _check_decode(cache, q * quiet, L, B, 2, got, idx, "f32", scale=scale)


def test_decode_missing_and_shared_pages(ssa):
    B, d, L = 16, 64, [100, 90, 60]
    cache = list(_cache("i8", d, B, 2, L, seed=5, poison=False))
    table = cache[5]
    table[1, :3] = table[0, :3]     # a shared prefix
    cache[4][1, :, :3] = cache[4][0, :, :3]
    q = torch.randn(3, 8, d, generator=torch.Generator().manual_seed(5))
    got, idx = _run_decode(ssa, cache, q, L, B, 1 << 20)
    _check_decode(cache, q, L, B, 1 << 20, got, idx, "f32")
    # a block without a page adds no keys: as if its keys were not there
    broken = list(cache)
    broken[5] = table.copy()
    broken[5][0, 2], broken[5][2, 1] = -1, 10 ** 6
    got2, _ = _run_decode(ssa, broken, q, L, B, 1 << 20)
    assert torch.equal(got2[1], got[1])
    Kv, Vv = (O.q8_values(_np(a), _np(b)) for a, b in ((cache[0], cache[1]), (cache[2], cache[3])))
    for b, gone in ((0, 2), (2, 1)):
        pos = [p for p in range(L[b]) if p // B != gone]
        for h in range(8):
            k, v = (x[table[b, np.array(pos) // B], h // 4, np.array(pos) % B] for x in (Kv, Vv))
            x = k @ _np(q)[b, h] / 8
            p = np.exp(x - x.max())
            ref = p @ v / p.sum()
            tol = np.abs(v).max() * (2 * np.abs(k * _np(q)[b, h]).sum(-1).max() / 8 * 8 * 2.0 ** -23
                                     + 2.0 ** -19)
            assert np.abs(_np(got2)[b, h] - ref).max() <= tol
    # no page at all: no key, zeros
    broken[5] = np.full_like(table, -1)
    got3, _ = _run_decode(ssa, broken, q, L, B, 1 << 20)
    assert (got3 == 0).all()


def test_decode_nan_scale_reaches_only_what_reads_it(ssa):
    B, d, L = 16, 64, [200, 200, 30]
    cache = list(_cache("e4m3", d, B, 2, L, seed=6))
    q = torch.randn(3, 4, d, generator=torch.Generator().manual_seed(6))
    clean, idx = _run_decode(ssa, cache, q, L, B, 3)
    left_out = next(j for j in range(1, 12) if j not in idx[0, 0].tolist())
    bad = [x.clone() if torch.is_tensor(x) else x for x in cache]
    bad[1][cache[5][0, left_out], 0] = float("nan")  # K of a block that is not chosen
    bad[3][cache[5][1, 0], 1] = float("nan")         # V of sequence 1's sink, head 1
    bad[1][cache[5][2, 1], 0] = float("nan")         # K of sequence 2's last block, head 0
    got, _ = _run_decode(ssa, bad, q, L, B, 3)
    nan = torch.isnan(got).all(-1).cpu()
    assert nan.tolist() == [[False] * 4, [False, False, True, True], [True, True, False, False]]
    assert torch.equal(got[~nan.to(DEV)], clean[~nan.to(DEV)])


def test_decode_on_another_stream_in_a_graph_and_twice_at_once(ssa):
    B, d = 64, 128
    L = [3000, 64, 1500]
    cache = _cache("e4m3", d, B, 2, L, seed=7)
    K, Ks, V, Vs, S = (x.to(DEV) for x in cache[:5])
    table, lens = _dev(cache[5]), _dev(np.asarray(L))
    g = torch.Generator().manual_seed(8)
    qs = [torch.randn(3, 8, d, generator=g).to(DEV, torch.bfloat16) for _ in range(2)]

    def call(q, topk=4, **kw):
        return ssa.ssa_decode_paged_q8(q, K, Ks, V, Vs, S, table, lens, B, topk, **kw)

    want = [call(q) for q in qs]
    whole = [call(q, topk=1 << 20) for q in qs]
    torch.cuda.synchronize()
    # two streams, each with the binding's own workspace; the current stream is another
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = []
        for q, s in zip(qs, streams):
            s.wait_stream(torch.cuda.current_stream())
            got.append(call(q, stream=s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # two graphs share one workspace; replays in turn, with new queries in between
    ws = torch.empty(ssa.ssa_decode_paged_q8_workspace_size(3, 8, 2, d, B, 4, table.shape[1]),
                     dtype=torch.uint8, device=DEV).fill_(255)
    q_in = qs[0].clone()
    outs, graphs = [], []
    for topk in (4, 1 << 20):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            call(q_in, topk=topk, workspace=None if topk > 4 else ws)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(call(q_in, topk=topk, workspace=ws))
        graphs.append(gr)
    for i in (1, 0, 1):
        q_in.copy_(qs[i])
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], want[i][0]) and torch.equal(outs[0][1], want[i][1])
        assert torch.equal(outs[1][0], whole[i][0])
    # both streams' calls in one graph, side by side
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs = []
        for q, s in zip(qs, streams):
            s.wait_stream(torch.cuda.current_stream())
            outs.append(call(q, stream=s))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            a[0].zero_(), a[1].zero_()


def test_results_on_another_stream_leave_the_current_ones_memory_alone(ssa):
    # memory freed behind a copy that the current stream has not run yet is not what a call
    # on another stream writes its results to
    B, d, n = 64, 128, 64
    L = [100] * n
    cache = _cache("e4m3", d, B, 2, L, seed=12)
    K, Ks, V, Vs, S = (x.to(DEV) for x in cache[:5])
    table, lens = _dev(cache[5]), _dev(np.asarray(L))
    q = torch.randn(n, 16, d, device=DEV, dtype=torch.bfloat16)
    have, want = _dev(np.zeros(n)), _dev(np.ones(n))
    ring, pool = _dev(np.arange(2 * n)), _dev(np.array([0, 2 * n]))
    ptable = torch.full((n, 4), -1, dtype=torch.int32, device=DEV)
    ref = ssa.ssa_decode_paged_q8(q, K, Ks, V, Vs, S, table, lens, B, 4)
    side = torch.cuda.Stream()
    for i in range(3):
        torch.cuda.synchronize()
        held = [torch.full_like(q, 7.), torch.full_like(ref[1], 7), torch.full((n * 8,), 7, device=DEV)]
        torch.cuda._sleep(20_000_000)  # cycles: some 10 ms
        kept = [x.clone() for x in held]
        del held
        got = ssa.ssa_decode_paged_q8(q, K, Ks, V, Vs, S, table, lens, B, 4, stream=side)
        plan = ssa.ssa_page_plan(have, want, ptable, ring, pool, B, 4 * n, stream=side)
        torch.cuda.synchronize()
        assert all((x == 7).all() for x in kept)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        assert plan[0].tolist() == [1] * n


@pytest.mark.parametrize("G,d,topk", [(4, 128, 1 << 20), (1, 64, 1 << 20), (8, 128, 5)])
def test_decode_repeats_bitwise(ssa, G, d, topk):
    # rows split between blocks: the block that joins a row's parts changes from run
    # to run, the order of the sums must not
    B, L = 32, [5000, 33, 2500, 700, 4100]
    cache = _cache("e4m3", d, B, 2, L, seed=33)
    K, Ks, V, Vs, S = (x.to(DEV) for x in cache[:5])
    table, lens = _dev(cache[5]), _dev(np.asarray(L))
    q = torch.randn(5, 2 * G, d, generator=torch.Generator().manual_seed(33)).to(DEV)
    for t in (torch.bfloat16, torch.float32):
        ref = None
        for i in range(200):
            out, _ = ssa.ssa_decode_paged_q8(q.to(t), K, Ks, V, Vs, S, table, lens, B, topk)
            if i % 7 == 0:  # another load on the GPU beside some of them
                torch.empty(1 << 22, device=DEV).fill_(i)
            ref = out if ref is None else ref
            assert torch.equal(out, ref)


# ------------------------------------------------------------------- together
def test_plan_and_append_in_a_graph_and_on_another_stream(ssa):
    # one captured step (plan of more than 8192 slots, append, decode), replayed
    # with other lengths and tokens in the same buffers, against eager calls
    B, d, Hkv, n, mb, cap = 16, 64, 2, 6, 300, 9000
    r = np.random.default_rng(40)
    pages = n * mb + 5
    order = r.permutation(pages)

    def fresh():
        return dict(K=torch.zeros(pages, Hkv, B, d, dtype=torch.int8, device=DEV),
                    V=torch.zeros(pages, Hkv, B, d, dtype=torch.int8, device=DEV),
                    Ks=torch.zeros(pages, Hkv, device=DEV), Vs=torch.zeros(pages, Hkv, device=DEV),
                    S=torch.zeros(n, Hkv, mb, d, device=DEV),
                    have=torch.zeros(n, dtype=torch.int32, device=DEV),
                    want=torch.zeros(n, dtype=torch.int32, device=DEV),
                    table=torch.full((n, mb), -1, dtype=torch.int32, device=DEV),
                    ring=_dev(order), pool=_dev(np.array([0, pages])),
                    k=torch.zeros(cap, Hkv, d, device=DEV, dtype=torch.bfloat16),
                    v=torch.zeros(cap, Hkv, d, device=DEV, dtype=torch.bfloat16),
                    q=torch.zeros(n, 4, d, device=DEV, dtype=torch.bfloat16))

    def step(s, stream=None):
        _, cu, slots, _ = ssa.ssa_page_plan(s["have"], s["want"], s["table"], s["ring"], s["pool"],
                                            B, cap, got=s["have"], pool_out=s["pool"],
                                            stream=stream)
        ssa.ssa_append_paged_q8(s["K"], s["Ks"], s["V"], s["Vs"], s["S"], slots, cu, s["have"],
                                s["k"], s["v"], B, stream=stream)
        return ssa.ssa_decode_paged_q8(s["q"], s["K"], s["Ks"], s["V"], s["Vs"], s["S"],
                                       s["table"], s["have"], B, 4, stream=stream)

    wants = [[3000, 17, 0, 900, 1, 4700], [3001, 18, 1500, 0, 2, 4701], [2990, 18, 1501, 700, 3, 0]]
    eager, captured, other = fresh(), fresh(), fresh()
    graph = torch.cuda.CUDAGraph()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        step(fresh())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step(captured)
    side = torch.cuda.Stream()
    for i, want in enumerate(wants):
        g = torch.Generator().manual_seed(41 + i)
        new = {x: torch.randn(eager[x].shape, generator=g).to(DEV, torch.bfloat16) for x in "kvq"}
        for s in (eager, captured, other):
            for x in "kvq":
                s[x].copy_(new[x])
            s["want"].copy_(_dev(np.array(want)))
        ref = step(eager)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        got = step(other, stream=side)
        torch.cuda.synchronize()
        assert eager["have"].tolist() == want
        for s, o in ((captured, out), (other, got)):
            for x in eager:
                assert torch.equal(eager[x], s[x]), x
            assert torch.equal(ref[0], o[0]) and torch.equal(ref[1], o[1])


def test_steps_in_a_row_equal_steps_one_by_one(ssa):
    """Every kernel starts while the one before it ends: 150 steps whose lengths, tables,
    lists and queries change each time give the same without a wait between any two
    calls as with one after each."""
    B, d, Hkv, n, mb, cap = 16, 128, 2, 24, 40, 6000
    r = np.random.default_rng(50)
    pages = n * mb // 2
    order = r.permutation(pages)
    have, wants = np.zeros(n, np.int64), []
    for i in range(150):
        w = np.where(r.random(n) < 0.8, have + 1, have + r.integers(-300, 400, n))
        wants.append(np.clip(w, 0, B * mb))
        have = wants[-1]  # (some rows are refused: the plan takes what comes)
    wants = [_dev(w) for w in wants]
    g = torch.Generator(device=DEV).manual_seed(51)
    k, v = (torch.randn(cap, Hkv, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(150, n, 8, d, generator=g, device=DEV).bfloat16()

    def run(topk, wait):
        K, V = (torch.zeros(pages, Hkv, B, d, dtype=torch.int8, device=DEV) for _ in range(2))
        Ks, Vs = (torch.zeros(pages, Hkv, device=DEV) for _ in range(2))
        S = torch.zeros(n, Hkv, mb, d, device=DEV)
        lens = torch.zeros(n, dtype=torch.int32, device=DEV)
        table = torch.full((n, mb), -1, dtype=torch.int32, device=DEV)
        ring, pool = _dev(order), _dev(np.array([0, pages]))
        q_in, outs = torch.empty_like(q[0]), []
        for i, want in enumerate(wants):
            q_in.copy_(q[i])
            wait()
            _, cu, slots, _ = ssa.ssa_page_plan(lens, want, table, ring, pool, B,
                                                cap if i % 3 else 9000, got=lens, pool_out=pool)
            wait()
            kk, vv = (x if i % 3 else torch.cat([x, x[:3000]]) for x in (k, v))
            ssa.ssa_append_paged_q8(K, Ks, V, Vs, S, slots, cu, lens, kk, vv, B)
            wait()
            outs.append(ssa.ssa_decode_paged_q8(q_in, K, Ks, V, Vs, S, table, lens, B, topk))
            wait()
        torch.cuda.synchronize()
        return outs, (K, Ks, V, Vs, S, lens, table, ring, pool)

    for topk in (3, 1 << 20):
        ref = run(topk, torch.cuda.synchronize)
        got = run(topk, lambda: None)
        for a, b in zip(ref[1], got[1]):
            assert torch.equal(a, b)
        for (a, ia), (b, ib) in zip(ref[0], got[0]):
            assert torch.equal(a, b) and torch.equal(ia, ib)


@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("i8", "f32")])
def test_serving_steps_plan_append_decode(ssa, fmt, dtype):
    """Prompts, decode steps, a rollback, a finished and a refused request, as a
    serving loop runs them; every step is checked against the oracle's."""
    B, d, Hq, Hkv, n, mb, pages, topk, cap = 16, 64, 4, 2, 5, 6, 16, 2, 160  # 16 pages: step 5 asks for 17
    r = np.random.default_rng(9)
    t = TORCH[dtype]
    K, V = (torch.zeros(pages, Hkv, B, d, device=DEV).to(TORCH[fmt]) for _ in range(2))
    Ks, Vs = (torch.zeros(pages, Hkv, device=DEV) for _ in range(2))
    S = torch.zeros(n, Hkv, mb, d, device=DEV)
    lens = torch.zeros(n, dtype=torch.int32, device=DEV)
    table = torch.full((n, mb), -1, dtype=torch.int32, device=DEV)
    ring, pool = _dev(r.permutation(pages)), _dev(np.array([0, pages]))
    rK, rKs, rV, rVs, rS = (_np(x) for x in (K, Ks, V, Vs, S))
    h, tb, rg, pl = lens.cpu().numpy(), table.cpu().numpy(), ring.cpu().numpy(), [0, pages]
    plans = [[70, 1, 40, 0, 16], [71, 2, 41, 0, 17], [72, 3, 42, 96, 18], [73, 4, 0, 96, 19],
             [68, 5, 0, 96, 20], [80, 6, 33, 96, 21], [81, 0, 34, 0, 22], [96, 80, 35, 0, 23]]
    refused = 0
    for step, want in enumerate(plans):
        k, v = (torch.randn(cap, Hkv, d, generator=torch.Generator().manual_seed(2 * step + i))
                .to(t) for i in range(2))
        q = torch.randn(n, Hq, d, generator=torch.Generator().manual_seed(100 + step)).to(t)
        _, cu, slots, _ = ssa.ssa_page_plan(lens, _dev(np.array(want)), table, ring, pool, B, cap,
                                            got=lens, pool_out=pool)
        ssa.ssa_append_paged_q8(K, Ks, V, Vs, S, slots, cu, lens, k.to(DEV), v.to(DEV), B)
        out, idx = ssa.ssa_decode_paged_q8(q.to(DEV), K, Ks, V, Vs, S, table, lens, B, topk)
        torch.cuda.synchronize()
        h, rcu, rsl, pl, tb, rg = O.page_plan(h, want, None, tb, rg, pl, B, cap)
        assert np.array_equal(lens.cpu().numpy(), h)
        refused += int((h != np.array(want)).sum())
        rK, rKs, rV, rVs, rS = O.append_paged_q8(rK, rKs, rV, rVs, rS, rsl, rcu, h, _np(k), _np(v),
                                                 B, fmt)
        for a, b in ((K, rK), (Ks, rKs), (V, rV), (Vs, rVs)):
            assert np.array_equal(_np(a), b)
        cache = (torch.from_numpy(rK), torch.from_numpy(rKs), torch.from_numpy(rV),
                 torch.from_numpy(rVs), S.cpu(), tb)
        _check_decode(cache, q, h, B, topk, out, idx, dtype)
    assert refused > 0 and pl[1] < pages
    assert ssa.ssa_device_error() == 0
