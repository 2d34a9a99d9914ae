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
- a bf16 result is rounded by half a step, 2^-8 of itself at most.

P's last bit: ``FLOOR`` of W for each key, the keys being those that a warp holds together.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_q8 import DEV, TORCH, _dev, _np

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
FLOOR = 2.0 ** -29


@pytest.fixture(scope="module")
def ssa():
    import block_sparse_top_summary_b200 as m
    m.load_library()
    return m


def _reference(q, K, Ks, V, Vs, table, L, B, scale, fmt):
    """Attention over the whole cache in 64 bits: ``(O, sum p |v| / l, W, e)`` of every head."""
    q, Kv, Vv = _np(q), O.q8_values(_np(K), _np(Ks)), O.q8_values(_np(V), _np(Vs))
    vs = _np(Vs)
    n, Hq, d = q.shape
    G = Hq // K.shape[1]
    out, mag = np.zeros_like(q), np.zeros_like(q)
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
                W[b, h] = (p * vs[page, g]).max() * O.QMAX[fmt] / l
                e[b, h] = scale * (np.abs(k) @ np.abs(q[b, h])).max() * (d / 16 + 4) * 2.0 ** -23
    return out, mag, W, e


def _check(got, ref, dtype, keys):
    """``keys``: the most that a warp holds together."""
    out, mag, W, e = ref
    tol = mag * (2 * e + 2.0 ** -19) + keys * FLOOR * W
    if dtype == "bf16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(out)
    err = np.abs(_np(got) - out)
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert np.all(err <= tol), (worst, _np(got)[worst], out[worst], tol[worst])


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
