"""Error of the 8-bit decode against 64 bits, by bounds that follow the row itself.

With p_t = exp(x_t - max x), l = sum p, and a row's largest weight W = max_t p_t vs_t QMAX / l
(vs_t: the scale of the block of V that key t lies in), all formed in 64 bits:

- a logit moves by at most e = A (d / 16 + 4) 2^-23, A = max_t scale sum_i |q_i k_ti| (q in two
  f16, d / 16 accumulations and the products with the scales, as in test_gpu_q8), which moves
  every p_t, and l, by a factor within exp(e): 2 e of sum p |v| / l;
- splitting P leaves 2^-22 of a p, ex2 and the factors less than 2^-21, and the sums of short
  runs (up to 2^4 slices of 16 keys a warp) and their joins less than 2^-20, all of sum p |v| / l;
  2^-19 in all;
- a p below the f16 parts' last bit is off by half of it;
- a p below 2^-126 is 0 in fp32 (ex2 flushes it; p refers to a maximum not above the row's, so
  no larger p is): what such keys add may be missing, the sum of their p |v| / l;
- a bf16 result is rounded by half a step, 2^-8 of itself at most, or 2^-134 where it is
  subnormal.

P's last bit: ``FLOOR`` of W for each key, the keys being those that a warp holds together.  Long
runs: sums of 32 slices, 64 products, each of which cuts off less than a step, 2^-23, of a sum that
grows evenly (half of 64 2^-23), 2^7 of those sums added with half a step each (2^-24 of a
growing sum, 2^-18) and the joins (2^-20): 2^-17 of sum p |v| / l.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_q8 import DEV, TORCH, _dev, _np

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
FLOOR = 2.0 ** -34  # half of f16's last bit, 2^-24, where the largest weight is at least 2^9


@pytest.fixture(scope="module")
def ssa():
    import block_sparse_top_summary_b200 as m
    m.load_library()
    return m


def _reference(q, K, Ks, V, Vs, table, L, B, scale, fmt):
    """Attention over the whole cache in 64 bits: ``(O, sum p |v| / l, W, e, sum p |v| / l of the p
    that fp32 may flush)`` of every head."""
    q, Kv, Vv = _np(q), O.q8_values(_np(K), _np(Ks)), O.q8_values(_np(V), _np(Vs))
    vs = _np(Vs)
    n, Hq, d = q.shape
    G = Hq // K.shape[1]
    out, mag, low = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    W, e = np.zeros((n, Hq, 1)), np.zeros((n, Hq, 1))
    for b in range(n):
        pos = np.arange(L[b])
        page, row = table[b, pos // B], pos % B
        for g in range(K.shape[1]):
            k, v = Kv[page, g, row], Vv[page, g, row]
            for h in range(g * G, (g + 1) * G):
                x = scale * (k @ q[b, h])
                p = np.exp(x - x.max())
                l = p.sum()
                out[b, h], mag[b, h] = p @ v / l, p @ np.abs(v) / l
                low[b, h] = (p * (p < 2.0 ** -125)) @ np.abs(v) / l
                W[b, h] = (p * vs[page, g]).max() * O.QMAX[fmt] / l
                e[b, h] = scale * (np.abs(k) @ np.abs(q[b, h])).max() * (d / 16 + 4) * 2.0 ** -23
    return out, mag, W, e, low


def _check(got, ref, dtype, keys):
    """``keys``: the most that a warp holds together."""
    out, mag, W, e, low = ref
    tol = mag * (2 * e + 2.0 ** -19) + keys * FLOOR * W + low
    if dtype == "bf16":
        tol = tol * (1 + 2.0 ** -8) + np.maximum(2.0 ** -8 * np.abs(out), 2.0 ** -134)
    err = np.abs(_np(got) - out)
    bad = np.argwhere(~(err <= tol))
    assert len(bad) == 0, [(len(bad), i.tolist(), _np(got)[tuple(i)], out[tuple(i)], tol[tuple(i)])
                           for i in bad[:3]]


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,n", [(128, 1), (64, 1), (128, 40)])
def test_probabilities_are_held_to_22_bits(ssa, fmt, dtype, d, n):
    # keys in pairs whose logits differ by one step of one coordinate and whose V are opposite:
    # a result far below the summed magnitudes, where a probability rounded to 11 bits shows
    B, Hkv, G, pages = 16, 2, 4, 6
    g = torch.Generator().manual_seed(d + n)
    K = torch.randint(-7, 8, (pages, Hkv, B, d), generator=g).float()
    K[:, :, 1::2] = K[:, :, 0::2]
    K[:, :, 1::2, 3] += 1
    V = torch.randint(100, 120, (pages, Hkv, B, d), generator=g).float()
    V = (V // 8 * 8) if fmt == "e4m3" else V
    V[:, :, 1::2] = -V[:, :, 0::2]
    K, V = K.to(TORCH[fmt]), V.to(TORCH[fmt])
    Ks, Vs = torch.full((pages, Hkv), 2.0 ** -4), torch.full((pages, Hkv), 2.0 ** -6)
    q = torch.randn(n, Hkv * G, d, generator=g).to(TORCH[dtype])
    L = [pages * B - 2 * (b % 5) for b in range(n)]
    table = np.stack([np.random.default_rng(b).permutation(pages) for b in range(n)])
    got, _ = ssa.ssa_decode_paged_q8(q.to(DEV), K.to(DEV), Ks.to(DEV), V.to(DEV), Vs.to(DEV), None,
                                     _dev(table), _dev(np.array(L)), B, 1 << 20)
    ref = _reference(q, K, Ks, V, Vs, table, L, B, 1 / math.sqrt(d), fmt)
    _check(got, ref, dtype, keys=B)


def _pool(fmt, exps, logits, B, Hkv, d, seed):
    """One page for each V exponent (None: all zeros, the least scale) and its logit (log2)."""
    g = torch.Generator().manual_seed(seed)
    n = len(exps)
    K = torch.randint(-7, 8, (n, Hkv, B, d), generator=g).float()
    V = torch.randn(n, Hkv, B, d, generator=g)
    V = (V * O.QMAX[fmt] / V.abs().amax(dim=(2, 3), keepdim=True))
    for i, x in enumerate(exps):
        if x is None:
            V[i] = 0
    V = V.round().to(TORCH[fmt]) if fmt == "i8" else V.to(TORCH[fmt])
    Vs = torch.tensor([2.0 ** (-126 if x is None else x) for x in exps])[:, None].expand(n, Hkv)
    Ks = torch.full((n, Hkv), 2.0 ** -5)
    if logits is not None:  # coordinate 0 alone, so that a q of ln 2 there gives the logit
        K.zero_()
        K[..., 0] = torch.tensor(logits, dtype=torch.float32)[:, None, None]
        Ks = torch.ones(n, Hkv)
    return K.to(TORCH[fmt]), Ks.contiguous(), V, Vs.float().contiguous()


def _decode(ssa, q, K, Ks, V, Vs, table, L, B, **kw):
    return ssa.ssa_decode_paged_q8(q.to(DEV), K.to(DEV), Ks.to(DEV), V.to(DEV), Vs.to(DEV), None,
                                   _dev(table), _dev(np.array(L)), B, 1 << 20, **kw)[0]


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,Hkv,G", [(6, 1, 4), (64, 4, 2)])
def test_values_of_unlike_scales(ssa, fmt, dtype, d, n, Hkv, G):
    # V scales from 2^-40 to 2^40 and pages of zeros, rising, falling, shuffled and drawn from some
    # of them, and K scales over three octaves: a row is a block's (6 rows: 8 slices a warp) or is
    # split between warps and blocks (64 rows of 4 heads: some 13 slices a warp)
    B, mb = 16, 90
    exps = [-40, -10, 0, 10, 40, None, 1, 2, 3, -3, -41, 41]
    K, Ks, V, Vs = _pool(fmt, exps, None, B, Hkv, d, seed=d + n)
    g = torch.Generator().manual_seed(n)
    Ks = Ks * torch.exp2(torch.randint(0, 4, Ks.shape, generator=g).float())
    q = (torch.randn(n, Hkv * G, d, generator=g) * 0.5).to(TORCH[dtype])
    order = np.argsort([-126 if x is None else x for x in exps])
    table = np.zeros((n, mb), int)
    for b in range(n):
        r = np.random.default_rng(b)
        some = r.choice(len(exps), size=2 + b % 5, replace=False) if b % 6 > 2 else np.arange(12)
        rank = np.isin(order, some)
        row = np.sort(r.integers(0, rank.sum(), mb))
        row = row[::-1] if b % 3 == 1 else r.permutation(row) if b % 3 == 2 else row
        table[b] = order[rank][row]
    L = [mb * B - 7 * (b % 4) for b in range(n)]
    got = _decode(ssa, q, K, Ks, V, Vs, table, L, B)
    _check(got, _reference(q, K, Ks, V, Vs, table, L, B, 1 / math.sqrt(d), fmt), dtype, keys=14 * B)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exps,logits", [
    ([0, -59, -118], [0, 0, 0]), ([0, -40, -80, -119], [0, 0, 0, 0]), ([-118, -59, 0], [0, 0, 0]),
    ([0, -61], [0, 104]), ([-61, 0], [0, -104]), ([0, 60], [0, -40]), ([60, 0], [0, 104]),
    ([100, -100], [0, 0]), ([0, 100], [0, -112]), ([100, 0, -100], [-112, -56, 0]),
    ([None, 20, None, 0], [0, -120, 24, -104]), ([None, 100], [0, -120]), ([None], [0])])
def test_one_warp_meets_values_of_scales_far_apart(ssa, fmt, dtype, exps, logits):
    # 96 pages to 12 warps, each in turn: what a warp has summed under one scale must neither
    # leave fp32's range nor hide what weighs more under another
    B, d, mb = 16, 64, 96
    K, Ks, V, Vs = _pool(fmt, exps, logits, B, 1, d, seed=len(exps))
    q = torch.zeros(1, 4, d)
    q[..., 0] = math.log(2)
    q[..., 1:] = torch.randn(1, 4, d - 1, generator=torch.Generator().manual_seed(1)) / 8
    q = q.to(TORCH[dtype])
    ways = [[min(i % 8, len(exps) - 1) for i in range(mb)],   # in order, then the last one
            [max(i % 8 - 8 + len(exps), 0) for i in range(mb)],  # the first one, then in order
            [i % len(exps) for i in range(mb)]]
    for way in ways:
        table = np.array([way])
        got = _decode(ssa, q, K, Ks, V, Vs, table, [mb * B], B, scale=1.0)
        ref = _reference(q, K, Ks, V, Vs, table, [mb * B], B, 1.0, fmt)
        _check(got, ref, dtype, keys=8 * B)


def _reference_of_pages(q, K, Ks, V, Vs, counts, scale, fmt):
    """As _reference for one KV head and rows that hold page i ``counts[i]`` times, whole; a key's
    e is its own here, and in place of it comes what it moves: sum p 2 e |v - O| / l."""
    q = _np(q)
    k = O.q8_values(_np(K), _np(Ks))[:, 0]
    v = O.q8_values(_np(V), _np(Vs))[:, 0]
    c = np.repeat(np.asarray(counts, float), k.shape[1])
    vs = np.repeat(_np(Vs)[:, 0], k.shape[1])
    k, v = k.reshape(-1, k.shape[-1]), v.reshape(-1, v.shape[-1])
    out, mag, move, W = [], [], [], []
    for h in range(q.shape[0]):
        x = scale * (k @ q[h])
        p = np.exp(x - x[c > 0].max()) * (c > 0)
        l = (c * p).sum()
        e = scale * (np.abs(k) @ np.abs(q[h])) * (q.shape[-1] / 16 + 4) * 2.0 ** -23
        out.append((c * p) @ v / l)
        mag.append((c * p) @ np.abs(v) / l)
        move.append((c * p * 2 * e) @ np.abs(v - out[-1]) / l)
        W.append([(p * vs).max() * O.QMAX[fmt] / l])
    return np.stack(out), np.stack(mag), np.array(W), np.stack(move)


ROWS, BLOCKS = 14, 16384  # 2^21 keys a row; 1034 slices, 16.6 K keys, a warp
KEYS = 16 * (ROWS * BLOCKS * 128 // 16 // (148 * 12) + 1)


def _check_long(got, ref):
    out, mag, W, move = ref
    tol = mag * 2.0 ** -17 + move + KEYS * FLOOR * W
    for row in _np(got):
        assert np.all(np.abs(row - out) <= tol), (np.abs(row - out) / tol).max()


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tail", [24.7, 27.3, 30.4])
def test_a_long_tail_behind_one_key(ssa, fmt, d, tail):
    # key 0 of every row, and 2^21 - 1 keys of 2^-tail of its p each whose V agree; half of the
    # coordinates of key 0 are 0, so that the tail alone shows there
    B = 128
    K = torch.zeros(2, 1, B, d)
    K[:, 0, :, 0] = -16
    K[0, 0, 0, 0] = 0
    V = torch.full((2, 1, B, d), 112.0)
    V[0, 0, 0, : d // 2] = 0
    K, V = K.to(TORCH[fmt]), V.to(TORCH[fmt])
    Ks, Vs = torch.ones(2, 1), torch.full((2, 1), 0.25)
    q = torch.zeros(ROWS, 2, d)
    q[..., 0] = tail * math.log(2) / 16
    table = np.ones((ROWS, BLOCKS))
    table[:, 0] = 0
    got = _decode(ssa, q, K, Ks, V, Vs, table, [BLOCKS * B] * ROWS, B, scale=1.0)
    _check_long(got, _reference_of_pages(q[0], K, Ks, V, Vs, [1, BLOCKS - 1], 1.0, fmt))


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("loud", [0.2, 2.0])
def test_long_runs_of_drawn_keys(ssa, fmt, d, loud):
    # V of one sign, so that sums grow; even logits, and ones that a few keys carry
    B, pages = 128, 64
    g = torch.Generator().manual_seed(d)
    K = torch.randint(-7, 8, (pages, 1, B, d), generator=g).to(TORCH[fmt])
    V = torch.randint(40, 128, (pages, 1, B, d), generator=g).float().to(TORCH[fmt])
    Ks, Vs = torch.full((pages, 1), 0.25), torch.exp2(torch.randint(-6, -3, (pages, 1), generator=g))
    q = (torch.randn(1, 2, d, generator=g) * loud).expand(ROWS, 2, d).contiguous()
    row = torch.randint(0, pages, (BLOCKS,), generator=g).numpy()
    table = np.stack([np.random.default_rng(b).permutation(row) for b in range(ROWS)])
    got = _decode(ssa, q, K, Ks, V, Vs.float(), table, [BLOCKS * B] * ROWS, B)
    ref = _reference_of_pages(q[0], K, Ks, V, Vs.float(), np.bincount(row, minlength=pages),
                              1 / math.sqrt(d), fmt)
    _check_long(got, ref)
