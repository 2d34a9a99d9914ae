"""Cases, plain forms and work counts of the serving step over a paged 8-bit KV cache.

Three operators, used one after the other in a serving step:

- plan:   pages, slot map and lengths of a batch of requests on the GPU
          (``ssa_page_plan``);
- append: new tokens of a ragged batch written into pages of 8-bit codes with a
          scale per page and KV head (``ssa_append_paged_q8``);
- decode: one query token per sequence against that cache, over the top-k
          blocks or all of them (``ssa_decode_paged_q8``).

A case is a dict; ``op`` names its operator.  ``run`` computes it in elementary
torch operations, or, where ``own`` is set, by the library's entry points.
Every pass can be repeated on its state: ``plan`` reads the lengths and the
pool's state from other tensors than it writes, and appending the same tokens
at the same places again changes nothing.
"""
import math
import zlib

import numpy as np
import torch

own = False

DEV = "cuda"
QMAX = {"e4m3": 448.0, "i8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
REAL = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # Latency of the host-free page bookkeeping of one decode step: every
        # request gets one token, one in 64 a new page.
        {"name": "plan_decode_256", "op": "plan", "batch": 256, "B": 64, "max_blocks": 1024,
         "grow": 1.0, "prompt": 1, "shrink": 0.0},
        # Continuous batching: decoding requests, admitted prompts of up to 8K
        # tokens, finished and rolled-back requests in one call.
        {"name": "plan_mixed_512", "op": "plan", "batch": 512, "B": 32, "max_blocks": 2048,
         "grow": 0.8, "prompt": 8192, "shrink": 0.1},
        # Admission of a machine's full load of prompts, about half a million tokens.
        {"name": "plan_prompts_1024", "op": "plan", "batch": 1024, "B": 16, "max_blocks": 1024,
         "grow": 0.5, "prompt": 8192, "shrink": 0.3},
        # One token for each of 64 decoding sequences (the decode workload's
        # batch and heads).
        {"name": "append_decode_64", "op": "append", "batch": 64, "tokens": 1, "Hkv": 8, "d": 128,
         "B": 64, "fmt": "e4m3", "dtype": "bf16"},
        # Ragged fp32 chunks, three KV heads, d = 64 and a block of 48.
        {"name": "append_odd_f32", "op": "append", "batch": 11, "tokens": 701, "Hkv": 3, "d": 64,
         "B": 48, "fmt": "i8", "dtype": "f32"},
        # Prompts of 37 sequences, about 64K tokens in all: a prefill chunk.
        {"name": "append_prompts_64k", "op": "append", "batch": 37, "tokens": 3500, "Hkv": 8,
         "d": 128, "B": 64, "fmt": "e4m3", "dtype": "bf16"},
        # The smallest call: one short sequence, all of its blocks.
        {"name": "decode_one_short", "op": "decode", "batch": 1, "L": 777, "ragged": False, "Hq": 4,
         "Hkv": 1, "d": 64, "B": 16, "topk": 1 << 20, "fmt": "i8", "dtype": "f32"},
        # One long conversation, top-k blocks: few rows, a long axis to route.
        {"name": "decode_one_128k_top32", "op": "decode", "batch": 1, "L": 131072, "ragged": False,
         "Hq": 32, "Hkv": 8, "d": 128, "B": 64, "topk": 32, "fmt": "e4m3", "dtype": "bf16"},
        # The same length read whole: the split over a long axis.
        {"name": "decode_one_128k_all", "op": "decode", "batch": 1, "L": 131072, "ragged": False,
         "Hq": 32, "Hkv": 8, "d": 128, "B": 64, "topk": 1 << 20, "fmt": "e4m3", "dtype": "bf16"},
        # A ragged batch of ordinary lengths read whole.
        {"name": "decode_ragged_32_all", "op": "decode", "batch": 32, "L": 16384, "ragged": True,
         "Hq": 32, "Hkv": 8, "d": 128, "B": 64, "topk": 1 << 20, "fmt": "i8", "dtype": "bf16"},
        # Blocks of 128, two query heads a group, ragged lengths, fp32 queries.
        {"name": "decode_ragged_24_top8_f32", "op": "decode", "batch": 24, "L": 30001,
         "ragged": True, "Hq": 8, "Hkv": 4, "d": 128, "B": 128, "topk": 8, "fmt": "e4m3",
         "dtype": "f32"},
        # The decode workload: 64 sequences of 65536 tokens, 32 / 8 heads, top-32.
        {"name": "decode_64x65536_top32", "op": "decode", "batch": 64, "L": 65536, "ragged": False,
         "Hq": 32, "Hkv": 8, "d": 128, "B": 64, "topk": 32, "fmt": "e4m3", "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode"])
    B = rng.choice([16, 32, 48, 64, 80, 96, 112, 128])
    if op == "plan":
        batch = _log(rng, 1, 4096)
        return {"op": op, "batch": batch, "B": B, "max_blocks": _log(rng, 8, 1024),
                "grow": rng.choice([0.3, 0.5, 0.8, 1.0]),
                "prompt": _log(rng, 1, max(1, min(8192, 500000 // batch))),
                "shrink": rng.choice([0.0, 0.1, 0.3])}
    d = rng.choice([64, 128])
    fmt = rng.choice(["e4m3", "i8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "append":
        batch = _log(rng, 1, 128)
        Hkv = rng.choice([1, 2, 3, 4, 5, 8])
        most = max(1, 65536 * 8 * 128 // (2 * batch * Hkv * d * (2 if dtype == "f32" else 1)))
        return {"op": op, "batch": batch, "tokens": _log(rng, 1, min(5000, most)), "Hkv": Hkv,
                "d": d, "B": B, "fmt": fmt, "dtype": dtype}
    Hkv = rng.choice([1, 2, 3, 4, 8])
    batch = _log(rng, 1, 64)
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    L = _log(rng, 1, max(1, min(131072, (1 << 29) // (batch * Hkv * d))))
    return {"op": op, "batch": batch, "L": L, "ragged": rng.random() < 0.6, "Hq": G * Hkv,
            "Hkv": Hkv, "d": d, "B": B, "topk": rng.choice([0, 1, 4, 8, 16, 32, 1 << 20]),
            "fmt": fmt, "dtype": dtype}


# --------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _host(seed):
    return np.random.RandomState(int(seed) % (1 << 31))


def _rows(case):
    """The draws behind a case's lengths: of the case alone, so that sizes and work
    are the same for every seed; a seed orders the rows."""
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return np.random.RandomState(zlib.crc32(text.encode()))


def _lengths(case, seed):
    """Cached tokens of each sequence of a decode case, on the host."""
    L, n = case["L"], case["batch"]
    lens = _rows(case).randint(max(1, L // 8), L + 1, n) if case["ragged"] else np.full(n, L)
    lens[0] = L
    return _host(seed).permutation(lens).astype(np.int64)


def _plan_rows(case, seed):
    """have, want and keep of every row of a plan case, on the host."""
    r = _rows(case)
    n, cap = case["batch"], case["B"] * case["max_blocks"]
    have = np.floor(np.exp(r.uniform(0, math.log(cap / 2 + 1), n))).astype(np.int64)
    kind = r.rand(n)
    grow = np.floor(np.exp(r.uniform(0, math.log(case["prompt"] + 1), n))).astype(np.int64)
    want = have + np.where(kind < case["grow"], np.maximum(1, np.minimum(grow, cap - have)), 0)
    fresh = (kind < case["grow"]) & (grow > 64)  # an admitted prompt starts from nothing
    have = np.where(fresh, 0, have)
    want = np.where(fresh, np.minimum(grow, cap), want)
    down = kind > 1.0 - case["shrink"]
    gone = r.rand(n) < 0.7  # finished, the others rolled back by a few tokens
    want = np.where(down, np.where(gone, 0, np.maximum(0, have - r.randint(1, 9, n))), want)
    keep = np.where(r.rand(n) < 0.2, have // case["B"] // 2, 0)  # a shared prefix
    order = _host(seed).permutation(n)
    return have[order], want[order], keep[order]


def _append_rows(case, seed):
    """Lengths before and new tokens of each sequence of an append case, on the host."""
    r = _rows(case)
    n, t = case["batch"], case["tokens"]
    new = np.full(n, 1) if t == 1 else r.randint(1, t + 1, n)
    have = r.randint(0, 4 * case["B"], n)
    if t > 1:
        have[r.rand(n) < 0.5] = 0
    order = _host(seed).permutation(n)
    return have[order].astype(np.int64), new[order].astype(np.int64)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV, torch.int32)


def _scale(amax, fmt):
    """The least power of two s with amax <= QMAX s, from exponent and mantissa."""
    m, e = torch.frexp(amax)
    top, bits = math.frexp(QMAX[fmt])
    e = torch.where(m > top, e + 1, e) - bits
    return torch.ldexp(torch.ones_like(amax), e.clamp(min=-126))


def _to_codes(x, fmt):
    """8-bit codes and power-of-two scales of blocks x [..., B, d] (one scale a block)."""
    scale = _scale(x.abs().amax(dim=(-1, -2)), fmt)
    y = x / scale[..., None, None]
    return (y.round() if fmt == "i8" else y).to(CODE[fmt]), scale


def _prepare_plan(case, seed):
    have, want, keep = _plan_rows(case, seed)
    n, B, mb = case["batch"], case["B"], case["max_blocks"]
    hb = -(-have // B)
    wb = -(-want // B)
    used, need = int(hb.sum()), int(np.maximum(wb - hb, 0).sum())
    pages = used + need + 64
    r = _host(seed + 1)
    order = r.permutation(pages)
    table = np.full((n, mb), -1)
    at = np.arange(mb)[None, :] < hb[:, None]
    table[at] = order[:used]
    free = pages - used
    head = int(r.randint(0, pages))
    ring = np.full(pages, -1)
    ring[(head + np.arange(free)) % pages] = order[used:]
    grow = int(np.maximum(want - have, 0).sum())
    return {"op": "plan", "B": B, "have": _i32(have), "want": _i32(want), "keep": _i32(keep),
            "table": _i32(table), "ring": _i32(ring), "pool": _i32(np.array([head, free])),
            "max_new": max(1, grow + grow // 16)}  # a captured batch is padded


def _prepare_append(case, seed):
    have, new = _append_rows(case, seed)
    n, B, Hkv, d, fmt = case["batch"], case["B"], case["Hkv"], case["d"], case["fmt"]
    g = _gen(seed)
    seqlens = have + new
    nb = -(-seqlens // B)
    mb = int(nb.max())
    r = _host(seed + 1)
    order = r.permutation(int(nb.sum()) + 8)
    cu = np.concatenate([[0], np.cumsum(new)])
    first = np.concatenate([[0], np.cumsum(nb)])
    seq = np.repeat(np.arange(n), new)
    pos = have[seq] + np.arange(cu[-1]) - cu[seq]
    slots = order[first[seq] + pos // B] * B + pos % B
    # the cache before the call: every page already holds tokens of one size or
    # another, so that some part-filled blocks have to grow their scale
    shape = (len(order), Hkv, B, d)
    loud = torch.exp2(torch.randint(-3, 1, shape[:2], generator=g, device=DEV))[..., None, None]
    K, Ks = _to_codes(torch.randn(shape, generator=g, device=DEV) * loud, fmt)
    V, Vs = _to_codes(torch.randn(shape, generator=g, device=DEV) * loud, fmt)
    t = REAL[case["dtype"]]
    k = torch.randn(int(cu[-1]), Hkv, d, generator=g, device=DEV)
    k *= torch.exp(0.5 * torch.randn(Hkv, d, generator=g, device=DEV))  # channels of unlike size
    v = torch.randn(int(cu[-1]), Hkv, d, generator=g, device=DEV)
    return {"op": "append", "B": B, "fmt": fmt, "K": K, "Ks": Ks, "V": V, "Vs": Vs,
            "S": torch.zeros(n, Hkv, mb, d, device=DEV), "slots": _i32(slots), "cu": _i32(cu),
            "seqlens": _i32(seqlens), "k": k.to(t), "v": v.to(t)}


def _prepare_decode(case, seed):
    """A cache whose keys carry, in top-k blocks of each KV head, a direction that
    its queries carry too: the structure that block routing is made for."""
    lens = _lengths(case, seed)
    n, B, Hkv, d, fmt = case["batch"], case["B"], case["Hkv"], case["d"], case["fmt"]
    G = case["Hq"] // Hkv
    g = _gen(seed)
    nb = -(-lens // B)
    mb = int(nb.max())
    first = np.concatenate([[0], np.cumsum(nb)])
    pages = int(first[-1]) + 3
    order = _host(seed + 1).permutation(pages)
    table = np.full((n, mb), -1)
    at = np.arange(mb)[None, :] < nb[:, None]
    table[at] = order[: first[-1]]
    K = torch.zeros(pages, Hkv, B, d, device=DEV, dtype=CODE[fmt])
    V = torch.zeros_like(K)
    Ks = torch.ones(pages, Hkv, device=DEV)
    Vs = torch.ones(pages, Hkv, device=DEV)
    S = torch.zeros(n, Hkv, mb, d, device=DEV)
    u = torch.randn(n, Hkv, d, generator=g, device=DEV)
    u *= 6.0 / u.norm(dim=-1, keepdim=True)
    tab = _i32(table).long()
    for b in range(n):
        nbb, last = int(nb[b]), int(lens[b] - 1) // B
        where = tab[b, :nbb]
        x = torch.randn(nbb, Hkv, B, d, generator=g, device=DEV)
        mine = torch.zeros(nbb, Hkv, device=DEV)
        if last > 1:
            score = torch.rand(last - 1, Hkv, generator=g, device=DEV)
            top = score.topk(min(case["topk"], last - 1), dim=0).indices + 1
            mine.scatter_(0, top, 1.0)
        x += (mine[..., None] * u[b])[:, :, None, :]
        k, ks = _to_codes(x, fmt)
        K.view(torch.int8)[where] = k.view(torch.int8)
        Ks[where] = ks
        S[b, :, :nbb] = (k.float().mean(dim=2) * ks[..., None]).transpose(0, 1)
        x.normal_(generator=g)
        v, vs = _to_codes(x, fmt)
        V.view(torch.int8)[where] = v.view(torch.int8)
        Vs[where] = vs
    q = torch.randn(n, Hkv, G, d, generator=g, device=DEV) + u[:, :, None, :]
    return {"op": "decode", "B": B, "topk": case["topk"], "K": K, "Ks": Ks, "V": V, "Vs": Vs, "S": S,
            "table": tab.int(), "seqlens": _i32(lens),
            "q": q.reshape(n, case["Hq"], d).to(REAL[case["dtype"]])}


def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append,
            "decode": _prepare_decode}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms
def _plan(s):
    B, table, ring, max_new = s["B"], s["table"], s["ring"], s["max_new"]
    n, mb = table.shape
    pages = ring.numel()
    have, want = s["have"].long(), s["want"].long()
    head, free = s["pool"].long().clamp(0, pages)
    hb, wb = (have + B - 1) // B, (want + B - 1) // B
    ok = (have >= 0) & (have <= mb * B) & (want >= 0) & (want <= mb * B)
    grow = torch.where(ok, (want - have).clamp(min=0), 0)
    need = torch.where(ok, (wb - hb).clamp(min=0), 0)
    C, P = grow.cumsum(0), need.cumsum(0)
    granted = ok & (grow > 0) & (C <= max_new) & ((need == 0) | (P <= free))
    down = ok & (want < have)
    got = torch.where(granted | down, want, have)
    # the blocks that a shrinking row gives back, and the ring's new end
    lo = torch.maximum(wb, torch.minimum(s["keep"].long().clamp(min=0), hb))
    back = torch.where(down, (hb - lo).clamp(min=0), 0)
    R = back.cumsum(0)
    taken = torch.where(granted, need, 0).sum()
    given = torch.minimum(R[-1], pages - free)
    pool = torch.stack([(head + taken) % pages, free - taken + given]).int()
    # slots
    cu = torch.cat([C.new_zeros(1), C.clamp(max=max_new)])
    t = torch.arange(max_new, device=DEV)
    b = torch.searchsorted(C, t, right=True).clamp(max=n - 1)
    pos = have[b] + t - (C - grow)[b]
    j = pos // B
    new = ring[(head + (P - need)[b] + j - hb[b]) % pages]
    page = torch.where(j >= hb[b], new, table[b, j.clamp(0, mb - 1)]).long()
    slots = torch.where(granted[b] & (t < C[-1]), page * B + pos % B, -1).int()
    # table and ring, in place
    col = torch.arange(mb, device=DEV)[None, :]
    rank = (R - back)[:, None] + col - lo[:, None]
    out = (down & (back > 0))[:, None] & (col >= lo[:, None]) & (col < hb[:, None])
    out &= rank < pages - free
    ring[((head + free + rank) % pages)[out]] = table[out]
    put = granted[:, None] & (col >= hb[:, None]) & (col < wb[:, None])
    fill = ring[(head + (P - need)[:, None] + col - hb[:, None]) % pages]
    table.copy_(torch.where(put, fill, table))
    return {"got": got.int(), "cu": cu.int(), "slots": slots, "pool": pool, "table": table,
            "ring": ring}


def _append_one(x, P, Ps, fmt, pages, inv, row, B):
    """Writes the rows x into the pages `pages[inv]`; what the pages' rows hold then."""
    n, Hkv, d = len(pages), x.shape[1], x.shape[2]
    full = torch.zeros(n * B, Hkv, d, device=DEV)
    full[inv * B + row] = x.float()
    fresh = torch.zeros(n * B, dtype=torch.bool, device=DEV)
    fresh[inv * B + row] = True
    full, fresh = full.view(n, B, Hkv, d).transpose(1, 2), fresh.view(n, 1, B, 1)
    start = torch.argmax(fresh.view(n, B).int(), dim=1)
    old = torch.arange(B, device=DEV)[None, :] < start[:, None]
    before = torch.where(start[:, None] > 0, Ps[pages], 0.0)
    scale = torch.maximum(before, _scale(full.abs().amax(dim=(2, 3)), fmt))
    had = P.view(torch.int8)[pages].view(P.dtype)
    y = torch.where(fresh, full / scale[..., None, None],
                    had.float() * (before / scale)[..., None, None])
    y = (y.round() if fmt == "i8" else y).to(P.dtype)
    y = torch.where(fresh | old.view(n, 1, B, 1), y.view(torch.int8), had.view(torch.int8))
    P.view(torch.int8)[pages] = y
    Ps[pages] = scale
    return y.view(P.dtype).float() * scale[..., None, None]


def _append(s):
    B, fmt, slots = s["B"], s["fmt"], s["slots"].long()
    t = torch.nonzero(slots >= 0).view(-1)
    pages, inv = torch.unique(slots[t] // B, return_inverse=True)
    row = slots[t] % B
    held = _append_one(s["k"][t], s["K"], s["Ks"], fmt, pages, inv, row, B)
    _append_one(s["v"][t], s["V"], s["Vs"], fmt, pages, inv, row, B)
    # summaries of the blocks whose last row was written
    end = torch.nonzero(row == B - 1).view(-1)
    cu = s["cu"].long()
    b = torch.searchsorted(cu, t[end], right=True) - 1
    j = (s["seqlens"].long()[b] - cu[b + 1] + t[end]) // B
    s["S"][b, :, j] = held[inv[end]].mean(dim=2)
    return {k: s[k] for k in ("K", "Ks", "V", "Vs", "S")}


def _select(s, kk):
    """Blocks that every (sequence, KV head) attends, ascending and padded with -1."""
    q, S, B = s["q"], s["S"], s["B"]
    n, Hkv, mb, d = S.shape
    last = (s["seqlens"].long() - 1) // B
    j = torch.arange(mb, device=DEV)
    cand = ((j >= 1) & (j < last[:, None]))[:, None].expand(n, Hkv, mb)
    if kk >= mb:
        pick = cand
    else:
        # scores in 64 bits: the order of near ones is what counts
        qbar = q.double().view(n, Hkv, -1, d).mean(dim=2)
        score = torch.einsum("bgjd,bgd->bgj", S.double(), qbar)
        score = torch.where(cand, score, -math.inf)
        rank = torch.argsort(score, dim=-1, descending=True, stable=True)[..., :kk]
        pick = torch.zeros_like(cand).scatter(-1, rank, True) & cand
    pick = pick | (j == 0) | (j == last[:, None])[:, None]
    width = min(kk, mb) + 2
    order = torch.where(pick, j, mb).sort(dim=-1).values
    order = torch.nn.functional.pad(order, (0, max(0, width - mb)), value=mb)[..., :width]
    return torch.where(order < mb, order, -1)


def _decode(s):
    q, B = s["q"], s["B"]
    n, Hkv, mb, d = s["S"].shape
    idx = _select(s, min(s["topk"], mb))
    page = torch.gather(s["table"].long()[:, None].expand(n, Hkv, mb), 2, idx.clamp(min=0))
    page = torch.where(idx >= 0, page, 0)
    head = torch.arange(Hkv, device=DEV)[None, :, None].expand_as(page)
    pos = idx[..., None] * B + torch.arange(B, device=DEV)
    seen = (idx[..., None] >= 0) & (pos < s["seqlens"].long()[:, None, None, None])
    k = s["K"].view(torch.int8)[page, head].view(s["K"].dtype).float()
    k = k * s["Ks"][page, head][..., None, None]
    x = torch.einsum("bghd,bgstd->bghst", q.float().view(n, Hkv, -1, d), k) / math.sqrt(d)
    del k
    x = torch.where(seen[:, :, None], x, -math.inf).flatten(3)
    p = torch.exp(x - x.amax(dim=-1, keepdim=True))
    p = (p / p.sum(dim=-1, keepdim=True)).view(n, Hkv, -1, *seen.shape[2:])
    v = s["V"].view(torch.int8)[page, head].view(s["V"].dtype).float()
    v = v * s["Vs"][page, head][..., None, None]
    o = torch.einsum("bghst,bgstd->bghd", p, v)
    return {"O": o.reshape(q.shape).to(q.dtype), "idx": idx.int()}


def _run_own(s):
    import block_sparse_top_summary_b200 as ssa

    if s["op"] == "plan":
        got, cu, slots, pool = ssa.ssa_page_plan(s["have"], s["want"], s["table"], s["ring"],
                                                 s["pool"], s["B"], s["max_new"], keep=s["keep"])
        return {"got": got, "cu": cu, "slots": slots, "pool": pool, "table": s["table"],
                "ring": s["ring"]}
    if s["op"] == "append":
        ssa.ssa_append_paged_q8(s["K"], s["Ks"], s["V"], s["Vs"], s["S"], s["slots"], s["cu"],
                                s["seqlens"], s["k"], s["v"], s["B"])
        return {k: s[k] for k in ("K", "Ks", "V", "Vs", "S")}
    O, idx = ssa.ssa_decode_paged_q8(s["q"], s["K"], s["Ks"], s["V"], s["Vs"], s["S"], s["table"],
                                     s["seqlens"], s["B"], s["topk"])
    return {"O": O, "idx": idx}


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plan, "append": _append, "decode": _decode}[state["op"]](state)


# ----------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass, the same for every seed."""
    B = case["B"]
    if case["op"] == "plan":
        have, want, _ = _plan_rows(case, 0)
        n = len(have)
        grow = int(np.maximum(want - have, 0).sum())
        pages = int(np.abs(-(-want // B) - -(-have // B)).sum())
        # lengths in and out, prefix sums, a slot a token, a table word and a
        # ring word a page
        return {"bytes": 4.0 * (5 * n + 1 + grow + grow // 16 + 2 * pages), "flops": 0.0}
    size = 2 if case["dtype"] == "bf16" else 4
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "append":
        have, new = _append_rows(case, 0)
        full = int(((have + new) // B - have // B).sum())
        blocks = int((-(-(have + new) // B) - have // B).sum())
        return {"bytes": float(2 * new.sum() * Hkv * d * (size + 1) + 4 * full * Hkv * d
                               + 8 * blocks * Hkv + 4 * new.sum()),
                "flops": float(4 * new.sum() * Hkv * d)}
    lens = _lengths(case, 0)
    last = (lens - 1) // B
    cand = np.maximum(last - 1, 0)
    some = cand > case["topk"]  # rows that have to be scored
    keys = np.where(some, (1 + case["topk"]) * B + lens - last * B, lens).sum()
    scored = np.where(some, cand, 0).sum()
    return {"bytes": float(2 * keys * Hkv * d + 8 * (keys // B) * Hkv + 4 * scored * Hkv * d
                           + 2 * len(lens) * case["Hq"] * d * size),
            "flops": float(4 * keys * case["Hq"] * d + 2 * scored * Hkv * d)}


# ------------------------------------------------------------ 64-bit definition
def _exact_plan(s):
    """The plan row by row."""
    B, max_new = s["B"], s["max_new"]
    have, want, keep, table, ring = (s[k].cpu().numpy().astype(np.int64)
                                     for k in ("have", "want", "keep", "table", "ring"))
    head, free = s["pool"].tolist()
    pages, old = len(ring), ring.copy()
    got, cu, slots = have.copy(), [0], np.full(max_new, -1)
    tokens = asked = taken = 0
    freed = []
    for b in range(len(have)):
        h, w = -(-have[b] // B), -(-want[b] // B)
        n, need = max(want[b] - have[b], 0), max(w - h, 0)
        start, first = tokens, asked
        tokens, asked = tokens + n, asked + need
        if n and tokens <= max_new and (not need or asked <= free):
            got[b] = want[b]
            table[b, h:w] = old[(head + first + np.arange(need)) % pages]
            taken += need
            pos = np.arange(have[b], want[b])
            slots[start:tokens] = table[b, pos // B] * B + pos % B
        elif want[b] < have[b]:
            got[b] = want[b]
            freed += table[b, max(w, min(keep[b], h)):h].tolist()
        cu.append(min(tokens, max_new))
    freed = freed[: pages - free]
    for i, p in enumerate(freed):
        ring[(head + free + i) % pages] = p
    pool = np.array([(head + taken) % pages, free - taken + len(freed)])
    return {"got": got, "cu": np.array(cu), "slots": slots, "pool": pool, "table": table,
            "ring": ring}


def _exact_append(s):
    """Page by page: the scale from the exponent of the largest value, codes by
    rounding in 64 bits, the summary as the mean of what the page holds."""
    B, fmt = s["B"], s["fmt"]
    slots = s["slots"].cpu().numpy()
    cu, lens = s["cu"].cpu().numpy(), s["seqlens"].cpu().numpy()
    out = {"S": s["S"].double()}
    for name, new in (("K", "k"), ("V", "v")):
        P, Ps = s[name].double(), s[name + "s"].double()
        for b in range(len(lens)):
            p0 = int(lens[b]) - int(cu[b + 1] - cu[b])
            x = s[new][int(cu[b]):int(cu[b + 1])].double()
            for j in range(p0 // B, (int(lens[b]) - 1) // B + 1):
                r0, r1 = max(p0 - j * B, 0), min(int(lens[b]) - j * B, B)
                page = int(slots[cu[b] + j * B + r0 - p0]) // B
                part = x[j * B + r0 - p0: j * B + r1 - p0].transpose(0, 1)
                amax = part.abs().amax(dim=(1, 2))
                e = torch.floor(torch.log2(amax / QMAX[fmt]))
                e = torch.where(amax > QMAX[fmt] * torch.exp2(e), e + 1, e)
                scale = torch.exp2(e.clamp(min=-126))
                if r0:
                    scale = torch.maximum(scale, Ps[page])
                    P[page, :, :r0] = _nearest(P[page, :, :r0] * (Ps[page] / scale)[:, None, None],
                                               fmt)
                P[page, :, r0:r1] = _nearest(part / scale[:, None, None], fmt)
                Ps[page] = scale
                if r1 == B and name == "K":
                    out["S"][b, :, j] = P[page].mean(dim=1) * scale[:, None]
        out[name], out[name + "s"] = (None if fmt == "i8" else P), Ps
    return out


def _nearest(y, fmt):
    """Nearest code value, ties to even, in 64 bits: steps of 1 (i8), or of 2^(e - 3)
    with 2^e <= |y|, not below 2^-9 (e4m3)."""
    if fmt == "i8":
        return torch.round(y)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_decode(s):
    """Sequence by sequence and head by head, the selected keys laid end to end."""
    B, q = s["B"], s["q"].double()
    n, Hkv, mb, d = s["S"].shape
    G = q.shape[1] // Hkv
    kk = min(s["topk"], mb)
    idx = np.full((n, Hkv, kk + 2), -1)
    O = torch.zeros_like(q)
    lens = s["seqlens"].tolist()
    for b in range(n):
        last = (lens[b] - 1) // B
        c = max(last - 1, 0)
        if c > kk:
            qb = q[b].view(Hkv, G, d).mean(dim=1)
            score = (s["S"][b, :, 1:last].double() @ qb[..., None])[..., 0].cpu().numpy()
            picks = [np.sort(np.lexsort((np.arange(c), -score[g]))[:kk]) + 1 for g in range(Hkv)]
        else:
            picks = [np.arange(1, last)] * Hkv
        for g in range(Hkv):
            sel = np.unique(np.concatenate([[0], picks[g], [last]])).astype(np.int64)
            idx[b, g, : len(sel)] = sel
            at = torch.from_numpy(sel).to(DEV)
            page = s["table"][b].long()[at]
            rows = (at[:, None] * B + torch.arange(B, device=DEV)).view(-1) < lens[b]
            k = (s["K"].view(torch.int8)[page, g].view(s["K"].dtype).double()
                 * s["Ks"][page, g].double()[:, None, None]).view(-1, d)[rows]
            v = (s["V"].view(torch.int8)[page, g].view(s["V"].dtype).double()
                 * s["Vs"][page, g].double()[:, None, None]).view(-1, d)[rows]
            O[b, g * G:(g + 1) * G] = torch.softmax(q[b, g * G:(g + 1) * G] @ k.T * d ** -0.5, -1) @ v
    return {"O": O, "idx": idx}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "decode": _exact_decode}[case["op"]](s)
