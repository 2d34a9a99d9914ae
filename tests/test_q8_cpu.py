"""Host-side checks of the page plan and the 8-bit paged cache that need no GPU:
the library's argument checks (every call below fails before a launch), and the
oracle's code arithmetic pinned against torch's e4m3 and closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from block_sparse_top_summary_b200 import abi

NULL = None
FAKE = ctypes.c_void_p(0x100000)  # never dereferenced
ODD = ctypes.c_void_p(0x100008)
ODD2 = ctypes.c_void_p(0x100002)


@pytest.fixture(scope="module")
def lib():
    return abi.load_library()


def _caller(fn, names, ok):
    def call(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[names.index(k)] = v
        return fn(*args)
    return call


def test_page_plan_rejections(lib):
    names = ["have", "want", "keep", "batch", "B", "table", "max_blocks", "num_pages", "ring",
             "pool", "pool_out", "got", "cu", "slots", "max_new", "stream"]
    call = _caller(lib.ssa_page_plan, names,
                   [FAKE, FAKE, NULL, 4, 64, FAKE, 16, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8,
                    NULL])
    for n in ("have", "want", "table", "ring", "pool", "pool_out", "got", "cu", "slots"):
        assert call(**{n: NULL}) == 1, n
        assert call(**{n: ODD2}) == 1, n
    assert call(keep=ODD2) == 1 and call(slots=ODD) == 1
    assert call(batch=0) == 1 and call(max_blocks=0) == 1 and call(num_pages=0) == 1
    assert call(max_new=-1) == 1 and call(B=0) == 1
    assert call(B=40) == 2 and call(B=144) == 2
    assert call(batch=8193) == 2 and call(max_new=(1 << 30) + 1) == 2
    assert call(max_blocks=1 << 26) == 2      # 2^32 tokens a row
    assert call(num_pages=1 << 26) == 2       # slots past 31 bits


def test_append_q8_rejections(lib):
    names = ["Kp", "Ks", "Vp", "Vs", "fmt", "S", "slots", "cu", "seqlens", "k", "v", "dt", "ts",
             "hs", "batch", "max_new", "Hkv", "d", "B", "max_blocks", "num_pages", "stream"]
    call = _caller(lib.ssa_append_paged_q8, names,
                   [FAKE, FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 256, 128, 2,
                    8, 2, 128, 64, 16, 32, NULL])
    for n in ("Kp", "Ks", "Vp", "Vs", "slots", "cu", "seqlens", "k", "v"):
        assert call(**{n: NULL}) == 1, n
        assert call(**{n: ODD2}) == 1, n
    for n in ("Kp", "Vp", "k", "v"):
        assert call(**{n: ODD}) == 1, n
    assert call(S=ODD) == 1
    assert call(fmt=2) == 1 and call(dt=7) == 1
    assert call(d=96) == 2 and call(B=40) == 2
    assert call(batch=0) == 1 and call(Hkv=0) == 1 and call(max_new=-1) == 1
    assert call(max_blocks=0) == 1 and call(num_pages=0) == 1
    assert call(ts=0) == 1 and call(hs=-128) == 1
    assert call(ts=260) == 1                  # not a multiple of 16 bytes
    assert call(ts=260, dt=0, fmt=9) == 1     # fp32: 260 is one, the format is not
    assert call(max_new=0) == 0               # no tokens: no work
    assert call(num_pages=1 << 26) == 2


def test_decode_q8_rejections(lib):
    names = ["q", "dt", "Kp", "Ks", "Vp", "Vs", "fmt", "S", "table", "max_blocks", "num_pages",
             "seqlens", "batch", "Hq", "Hkv", "d", "B", "topk", "scale", "O", "idx", "ws",
             "ws_bytes", "stream"]
    need = abi.ssa_decode_paged_q8_workspace_size(2, 8, 2, 128, 64, 4, 64)
    assert need > 0 and need % 256 == 0
    call = _caller(lib.ssa_decode_paged_q8, names,
                   [FAKE, 1, FAKE, FAKE, FAKE, FAKE, 0, FAKE, FAKE, 64, 200, FAKE, 2, 8, 2, 128,
                    64, 4, 0.088, FAKE, NULL, FAKE, need, NULL])
    for n in ("q", "Kp", "Ks", "Vp", "Vs", "S", "table", "seqlens", "O", "ws"):
        assert call(**{n: NULL}) == 1, n
        assert call(**{n: ODD2}) == 1, n
    for n in ("q", "Kp", "Vp", "S", "O", "ws"):
        assert call(**{n: ODD}) == 1, n
    assert call(S=NULL, topk=61) == 1         # 62 candidates at most
    assert call(idx=ODD2) == 1
    assert call(ws=ctypes.c_void_p(0x100010)) == 1
    assert call(ws_bytes=need - 1) == 1
    assert call(fmt=2) == 1 and call(dt=2) == 1
    assert call(Hq=7) == 1 and call(Hq=18) == 2
    assert call(topk=-1) == 1 and call(batch=0) == 1
    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1
    assert call(d=32) == 2 and call(B=24) == 2
    assert call(max_blocks=16385) == 2
    # slices of the batch, and of the batch and its heads, past what the kernels count
    assert call(max_blocks=16384, batch=40000) == 2
    assert call(max_blocks=16384, batch=30000, Hq=4096, Hkv=4096, topk=1 << 30) == 2
    assert call(max_blocks=16384, batch=30000, Hq=4096, Hkv=4096, topk=1 << 30, q=NULL) == 2
    n = ctypes.c_size_t(0)
    f = lib.ssa_decode_paged_q8_workspace_size
    assert f(2, 7, 2, 128, 64, 4, 64, ctypes.byref(n)) == 1
    assert f(2, 8, 2, 128, 64, 4, 64, NULL) == 1
    # a few short rows read whole need none; lists are kept only where blocks can be left out
    assert abi.ssa_decode_paged_q8_workspace_size(2, 8, 2, 128, 64, 62, 24) == 0
    assert abi.ssa_decode_paged_q8_workspace_size(2, 8, 2, 128, 64, 62, 25) > 0
    assert abi.ssa_decode_paged_q8_workspace_size(75, 8, 2, 128, 64, 62, 24) > 0
    assert abi.ssa_decode_paged_q8_workspace_size(2, 8, 2, 128, 64, 4, 24) > 0
    assert abi.ssa_decode_paged_q8_workspace_size(64, 32, 8, 128, 64, 1 << 30, 16384) < 16 << 20


def test_words_are_the_calls_arguments(lib):
    """The packed forms refuse and accept what the calls do, word by word."""
    fake = FAKE.value
    plan = [fake] * 3 + [4, 64, fake, 8, 40] + [fake] * 6 + [10, 0]
    append = [fake] * 4 + [0] + [fake] * 6 + [1, 256, 128, 2, 10, 2, 128, 64, 8, 40, 0]
    need = abi.ssa_decode_paged_q8_workspace_size(2, 8, 2, 128, 64, 4, 64)
    decode = [fake, 1] + [fake] * 4 + [0, fake, fake, 64, 200, fake, 2, 8, 2, 128, 64, 4, 0.088,
                                       fake, 0, fake, need, 0]
    assert lib.ssa_page_plan_words(None) == 1
    # one argument at a time: what each call answers to a null pointer, an odd one, a number
    # out of its range or its type's
    for name, pack, ok in (("ssa_page_plan", abi._plan_words, plan),
                           ("ssa_append_paged_q8", abi._append_words, append),
                           ("ssa_decode_paged_q8", abi._decode_words, decode)):
        words, call = getattr(lib, name + "_words"), getattr(lib, name)
        for i, v in enumerate(ok):
            bad = ([-1.0] if isinstance(v, float) else [0, fake + 2] if v == fake
                   else [0] if v == need else [-5])
            for x in bad:
                a = ok[:i] + [x] + ok[i + 1:]
                if i == len(ok) - 1 or (name, i) in OPTIONAL and x == 0:
                    continue  # (these would launch)
                want = call(*a)
                assert want in (1, 2), (name, i, x)
                assert words(pack(*a)) == want, (name, i, x)
            if 0 < v < fake and not isinstance(v, float) and (name, i) not in WIDE:
                a = ok[:i] + [v + (1 << 32)] + ok[i + 1:]
                assert words(pack(*a)) == 1, (name, i)


# arguments that may be null, and those of 64 bits
OPTIONAL = {("ssa_page_plan", 2), ("ssa_append_paged_q8", 5), ("ssa_decode_paged_q8", 20)}
WIDE = {("ssa_append_paged_q8", 12), ("ssa_append_paged_q8", 13), ("ssa_decode_paged_q8", 22)}


def test_binding_refuses_what_is_not_on_a_gpu(monkeypatch):
    monkeypatch.setattr(abi, "_device", lambda: 0)
    K, s = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        abi._q8_cache(K.view(torch.uint8), s, K, s, None, 16, 0, 1, 4)
    with pytest.raises(ValueError, match="Kp must be a CUDA tensor"):
        abi.ssa_decode_paged_q8(torch.zeros(1, 4, 64), K, s, K, s, None, i[None], i, 16, 9)
    with pytest.raises(ValueError, match="Kp must be a CUDA tensor"):
        abi.ssa_append_paged_q8(K, s, K, s, None, i, i, i, s, s, 16, max_blocks=1)
    with pytest.raises(ValueError, match="max_blocks"):
        abi.ssa_append_paged_q8(K, s, K, s, None, i, i, i, s, s, 16)
    with pytest.raises(ValueError, match="have must be a CUDA tensor"):
        abi.ssa_page_plan(i, i, i[None], i, torch.zeros(2, dtype=torch.int32), 16, 4)


def test_oracle_codes_match_torch_e4m3_and_closed_forms():
    # every e4m3 value, and points on, below and above the middle of each pair
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mid = (v[1:] + v[:-1]) / 2
    pts = np.concatenate([v, mid, mid * (1 - 1e-6), mid * (1 + 1e-6)])
    pts = np.concatenate([pts, -pts])
    want = torch.from_numpy(pts).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.nearest_code(pts, "e4m3"), want)
    assert np.array_equal(O.nearest_code([0.5, 1.5, -2.5, 126.4, -127.0], "i8"),
                          [0.0, 2.0, -2.0, 126.0, -127.0])
    for fmt, top in O.QMAX.items():
        for e in (-126, -40, 0, 7, 100):
            assert O.q8_scale(top * 2.0 ** e, fmt) == 2.0 ** e
            if e > -126:
                assert O.q8_scale(top * 2.0 ** e * (1 - 1e-7), fmt) == 2.0 ** e
            assert O.q8_scale(top * 2.0 ** e * (1 + 1e-7), fmt) == 2.0 ** (e + 1)
        assert O.q8_scale(0.0, fmt) == 2.0 ** -126


def test_oracle_plan_on_a_case_done_by_hand():
    # B = 16, 4 rows; ring of 6 pages, 3 free from entry 5 on: pages 9, 7, 8
    table = np.array([[1, 2, -1], [3, -1, -1], [4, 5, 6], [-1, -1, -1]])
    ring = np.array([7, 8, 0, 0, 0, 9])
    got, cu, slots, pool, t2, r2 = O.page_plan(
        [17, 16, 40, 0], [18, 17, 16, 33], [0, 0, 0, 0], table, ring, [5, 3], 16, 8)
    assert got.tolist() == [18, 17, 16, 0]        # row 3 wants 33 tokens: 8 fit
    assert cu.tolist() == [0, 1, 2, 2, 8]
    assert slots.tolist() == [2 * 16 + 1, 9 * 16, -1, -1, -1, -1, -1, -1]
    assert t2[1].tolist() == [3, 9, -1] and t2[3].tolist() == [-1, -1, -1]
    assert pool.tolist() == [0, 4]                # one taken, pages 5 and 6 back
    assert [r2[(0 + i) % 6] for i in range(4)] == [7, 8, 5, 6]
