"""What is measured of the window-plus-first-tokens attention and of the 4-bit
paged cache: cases, inputs, a plain form of each operator in elementary torch
operations, and the values in 64 bits.

Operators
  fwd     sliding window attention whose first `first` tokens of each document
          stay visible (forward, packed documents, per-head sink logit)
  bwd     its backward: gradients of q, k, v and of the sink
  append  quantise new key / value rows to 4 bits, write them into the pages of
          their sequences, and read the same rows back as values
  decode  one query token per sequence over the paged 4-bit cache

With ``own`` false ``run`` computes the plain form (fp32, any tree); with
``own`` true it makes the library's calls.
"""

import math
import random

import torch

own = False

GROUP = 32  # elements that share one scale of the 4-bit cache


# ------------------------------------------------------------------ cases
def listed():
    mla = dict(H=64, dk=576, dv=512, dtype="bf16")
    return [
        # the tiny fp32 workload: 4 heads, window 32, launch latency counts
        dict(name="fwd_tiny_f32", op="fwd", T=256, docs=1, split=0, H=4, dk=64, dv=48,
             dtype="f32", window=32, first=4, sink=True),
        # the main training workload, one document
        dict(name="fwd_main", op="fwd", T=4096, docs=1, split=0, window=512, first=4, sink=True, **mla),
        # packed documents of ragged lengths
        dict(name="fwd_packed6", op="fwd", T=16384, docs=6, split=1, window=512, first=16,
             sink=True, **mla),
        # the narrow window layer of the sweep, a wide window
        dict(name="fwd_narrow_w1024", op="fwd", T=8192, docs=2, split=2, H=64, dk=192, dv=128,
             dtype="bf16", window=1024, first=64, sink=False),
        # backward of a short ragged batch
        dict(name="bwd_short", op="bwd", T=333, docs=3, split=3, window=64, first=5, sink=True, **mla),
        # backward of the main training workload
        dict(name="bwd_main", op="bwd", T=4096, docs=1, split=0, window=512, first=4, sink=True, **mla),
        # one new token for each of 64 running sequences
        dict(name="append_step64", op="append", S=64, new=1, old=2048, split=4, dk=576, dv=512,
             page=64, dtype="bf16"),
        # a prompt batch enters the cache; values are the latent part of the keys
        dict(name="append_prompt16k", op="append", S=6, new=4096, old=0, split=5, dk=576, dv=0,
             page=64, dtype="bf16"),
        # one short sequence: latency
        dict(name="decode_one_short", op="decode", S=1, length=777, split=6, H=64, dk=576, dv=512,
             alias=True, page=64, window=0, first=0, sink=False, dtype="bf16"),
        # a serving batch of ragged lengths, values = latent part of the keys
        dict(name="decode_batch64", op="decode", S=64, length=8192, split=7, H=64, dk=576, dv=512,
             alias=True, page=64, window=0, first=0, sink=True, dtype="bf16"),
        # a few long sequences with a value plane of their own
        dict(name="decode_long4", op="decode", S=4, length=65536, split=8, H=64, dk=576, dv=512,
             alias=False, page=128, window=0, first=0, sink=True, dtype="bf16"),
        # streaming: many long sequences, first tokens and window only, heads split over GPUs
        dict(name="decode_stream192", op="decode", S=192, length=16384, split=9, H=16, dk=576, dv=512,
             alias=True, page=16, window=1024, first=4, sink=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "bwd", "append", "decode"))
    split = rng.randrange(1 << 20)
    if op in ("fwd", "bwd"):
        if rng.random() < 0.2:  # small fp32
            return dict(op=op, T=_log(rng, 33, 400), docs=rng.randint(1, 3), split=split,
                        H=rng.choice((1, 2, 3, 4)), dk=64, dv=48, dtype="f32",
                        window=_log(rng, 1, 48), first=_log(rng, 1, 16), sink=rng.random() < 0.7)
        dk, dv = rng.choice(((576, 512), (576, 512), (512, 512), (192, 128)))
        T = _log(rng, 40, 8192 if op == "fwd" else 4096)
        return dict(op=op, T=T, docs=rng.randint(1, 6), split=split, H=64, dk=dk, dv=dv,
                    dtype="bf16", window=_log(rng, 8, 512), first=_log(rng, 1, 96),
                    sink=rng.random() < 0.7)
    dk, dv = rng.choice(((576, 512), (576, 512), (512, 512), (192, 128)))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        S = _log(rng, 1, 128)
        return dict(op=op, S=S, new=_log(rng, 1, 16384 // S), old=_log(rng, 1, 1024), split=split,
                    dk=dk, dv=rng.choice((0, dv)), page=page, dtype=rng.choice(("bf16", "bf16", "f32")))
    S = _log(rng, 1, 256)
    windowed = rng.random() < 0.3
    return dict(op=op, S=S, length=_log(rng, 1, min(65536, 262144 // S)), split=split,
                H=rng.choice((16, 32, 64, 64, 128)), dk=dk, dv=dv, alias=rng.random() < 0.5,
                page=page, window=_log(rng, 16, 2048) if windowed else 0,
                first=_log(rng, 1, 64) if windowed else 0, sink=rng.random() < 0.5, dtype="bf16")


def _doc_lengths(case):
    """Ragged document lengths that sum to T, from the case alone."""
    T, n = case["T"], min(case["docs"], case["T"])
    cuts = sorted(random.Random(case["split"]).sample(range(1, T), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def _seq_lengths(case):
    """Lengths of the cached sequences; the first one has the full length."""
    r, n = random.Random(case["split"]), case["length"]
    return [n] + [r.randint(max(1, n // 4), n) for _ in range(case["S"] - 1)]


def _append_lengths(case):
    """(rows already in the cache, new rows) of each sequence."""
    r = random.Random(case["split"])
    new = [case["new"]] + [r.randint(max(1, case["new"] // 4), case["new"]) for _ in range(case["S"] - 1)]
    return [r.randint(0, case["old"]) for _ in range(case["S"])], new


def _row_bytes(width):
    return width // 2 + 4 * -(-width // 128)


def work(case):
    op, isz = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("fwd", "bwd"):
        H, dk, dv, T, span = case["H"], case["dk"], case["dv"], case["T"], case["window"] + case["first"]
        pairs = sum(n * (n + 1) // 2 if n <= span else span * (span + 1) // 2 + (n - span) * span
                    for n in _doc_lengths(case))
        kv = T * (dk + dv) * isz
        if op == "fwd":
            return {"bytes": T * H * (dk + dv) * isz + kv + 4 * T * H, "flops": 2 * H * pairs * (dk + dv)}
        return {"bytes": T * H * (2 * dk + 2 * dv) * isz + 2 * kv + 4 * T * H,
                "flops": 2 * H * pairs * (3 * dk + 2 * dv)}
    if op == "append":
        n = sum(_append_lengths(case)[1])
        # rows in, 4-bit rows written and read again, values out
        return {"bytes": sum(n * (w * (isz + 2) + 2 * (w // 2 + w // 32)) for w in (case["dk"], case["dv"]) if w),
                "flops": 0}
    span = case["window"] + case["first"] if case["window"] else 1 << 60
    keys = sum(min(n, span) for n in _seq_lengths(case))
    S, H, dk, dv = case["S"], case["H"], case["dk"], case["dv"]
    row = dk // 2 + dk // 32 + (0 if case["alias"] else dv // 2 + dv // 32)
    return {"bytes": keys * row + S * H * (dk + dv) * isz + 4 * S * H, "flops": 2 * H * keys * (dk + dv)}


# ------------------------------------------------------------------ the 4-bit format
# A group of 32 elements has one byte of scale, the upper bits of a half without
# sign (5 exponent and 3 mantissa bits): the smallest such number that is not
# below max|x| / 7.  Codes are rint(x / scale) + 8.  A page holds, for each
# group, `page` x 16 bytes of codes, then for each four groups `page` x 4 bytes
# of scales.  In a 32-bit word bits 4k.. hold element 2k, bits 16+4k.. element 2k+1.
def _quantise(x):
    """x [n, D] -> (codes [n, G, 32] in 1..15, scales [n, G]) of the plain form,
    in 64 bits: quotients next to a border between two scales or codes."""
    g = x.double().reshape(x.shape[0], -1, GROUP)
    r = g.abs().amax(-1) / 7.0
    _, e = torch.frexp(r)
    step = torch.ldexp(torch.ones_like(r), torch.clamp(e, min=-13) - 4)
    scale = torch.clamp(torch.ceil(r / step) * step, max=61440.0)
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = torch.clamp(torch.round(g / safe.unsqueeze(-1)), -7, 7)
    return (code + 8).to(torch.uint8), scale


def _pack(code, scale):
    """-> (16 bytes of codes [n, G, 16], byte of scale [n, G])"""
    n, G, _ = code.shape
    c = code.reshape(n, G, 4, 4, 2).to(torch.int32)  # word, k, parity
    word = c[..., 0].new_zeros(n, G, 4, 4)
    # byte b of a word: elements 2k with k = 2b, 2b + 1 for b < 2, then the odd ones
    word[..., 0] = c[..., 0, 0] | c[..., 1, 0] << 4
    word[..., 1] = c[..., 2, 0] | c[..., 3, 0] << 4
    word[..., 2] = c[..., 0, 1] | c[..., 1, 1] << 4
    word[..., 3] = c[..., 2, 1] | c[..., 3, 1] << 4
    byte = (scale.half().view(torch.int16) >> 7).to(torch.uint8)
    return word.to(torch.uint8).reshape(n, G, 16), byte


def _values(codes, byte):
    """16 bytes of codes [..., G, 16] and a byte of scale [..., G] -> fp32 [..., G * 32]"""
    b = codes.reshape(*codes.shape[:-1], 4, 4)
    nib = torch.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], 8)  # e0 e2 e4 e6 e1 e3 e5 e7
    nib = nib.reshape(*b.shape[:-1], 2, 4).transpose(-1, -2)          # pairs (even, odd)
    scale = (byte.to(torch.int16) << 7).view(torch.float16).float()
    v = (nib.reshape(*codes.shape[:-1], GROUP).float() - 8) * scale.unsqueeze(-1)
    return v.reshape(*codes.shape[:-2], -1)


def _planes(cache, width, page):
    """Views of a cache [pages, bytes]: codes [pages, G, page, 16], scales [pages, Q, page, 4]."""
    G = width // GROUP
    n = cache.shape[0]
    return (cache[:, :G * page * 16].view(n, G, page, 16),
            cache[:, G * page * 16:].view(n, -(-G // 4), page, 4))


def _write(cache, width, page, pages, slots, x):
    G = width // GROUP
    code, byte = _pack(*_quantise(x))
    c, s = _planes(cache, width, page)
    c[pages, :, slots] = code
    full = torch.zeros((x.shape[0], 4 * -(-G // 4)), dtype=torch.uint8, device=x.device)
    full[:, :G] = byte
    s[pages, :, slots] = full.view(x.shape[0], -1, 4)


def _gather(cache, width, page, pages, slots):
    """Values fp32 [..., width] of the rows (pages, slots)."""
    G = width // GROUP
    c, s = _planes(cache, width, page)
    codes = c[pages, :, slots]
    scales = s[pages, :, slots].reshape(*pages.shape, -1)[..., :G]
    return _values(codes, scales)


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _table(lengths, page, gen, dev):
    """Pages of each sequence, in no order, from a pool with some to spare."""
    need = [-(-n // page) for n in lengths]
    pool = sum(need) + 7
    perm = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((len(lengths), max(1, max(need))), dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, pool


def prepare(case, seed):
    dev, dt = "cuda", _dtype(case)
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def randn(*shape, dtype=dt):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    st = dict(case=case)
    if case["op"] in ("fwd", "bwd"):
        T, H, dk, dv = case["T"], case["H"], case["dk"], case["dv"]
        lens = _doc_lengths(case)
        st["q"], st["k"], st["v"] = randn(T, H, dk), randn(T, dk), randn(T, dv)
        st["sink"] = randn(H, dtype=torch.float32) if case["sink"] else None
        st["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
        st["maxlen"] = max(lens)
        if case["op"] == "bwd":  # what a training step kept of its forward pass
            st["dout"] = randn(T, H, dv)
            st["out"], st["lse"] = _fwd(st)
        return st
    page, dk, dv = case["page"], case["dk"], case["dv"]
    if case["op"] == "append":
        old, new = _append_lengths(case)
        total = [a + b for a, b in zip(old, new)]
        n = sum(new)
        st["k"] = randn(n, dk)
        st["v"] = randn(n, dv) if dv else None
    else:
        total = _seq_lengths(case)
    st["table"], pool = _table(total, page, gen, dev)
    st["lens"] = torch.tensor(total, device=dev, dtype=torch.int32)
    st["maxlen"] = max(total)
    for name, width in (("kc", dk), ("vc", 0 if case.get("alias") else dv)):
        st[name] = torch.zeros((pool, page * _row_bytes(width)), dtype=torch.uint8, device=dev) if width else None
    if case["op"] == "append":
        st["cu"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
        return st
    st["q"] = randn(case["S"], case["H"], dk)
    st["sink"] = randn(case["H"], dtype=torch.float32) if case["sink"] else None
    every = torch.arange(pool * page, device=dev)
    for name, width in (("kc", dk), ("vc", 0 if case["alias"] else dv)):
        for part in every.split(1 << 17) if width else ():
            _write(st[name], width, page, part // page, part % page, randn(len(part), width, dtype=torch.bfloat16))
    return st


# ------------------------------------------------------------------ plain forms
CHUNK = 128  # queries that share one band of keys in the plain form


def _bands(st):
    """Key indices and masks: a band of keys per chunk of queries, and the first
    tokens of each query's document that lie before its window."""
    case, cu, T = st["case"], st["cu"].long(), st["q"].shape[0]
    W, F, dev = min(case["window"], st["maxlen"]), min(case["first"], st["maxlen"]), st["q"].device
    n = -(-T // CHUNK)
    t = torch.arange(n * CHUNK, device=dev)
    bos = cu[torch.searchsorted(cu[1:].contiguous(), t.clamp(max=T - 1), right=True)]
    lo = torch.maximum(bos, t - W + 1)
    band = torch.arange(n, device=dev)[:, None] * CHUNK - (W - 1) + torch.arange(CHUNK + W - 1, device=dev)
    tt, ll = t.view(n, CHUNK, 1), lo.view(n, CHUNK, 1)
    bmask = (band[:, None] >= ll) & (band[:, None] <= tt) & (tt < T)
    fidx = bos[:T, None] + torch.arange(F, device=dev)
    return n, band.clamp(0, T - 1), bmask, fidx.clamp(max=T - 1), fidx < lo[:T, None]


def _padded(x, n):
    x = x.float()
    return torch.cat((x, x.new_zeros((n * CHUNK - x.shape[0],) + x.shape[1:])))


def _dots(x, rows, n, band, fidx):
    """<x[t, h], rows[j]> over the band [n * CHUNK, H, span] and the first tokens [T, H, F]."""
    T, H, d = x.shape
    b = torch.matmul(_padded(x, n).view(n, CHUNK * H, d), rows[band].transpose(1, 2))
    return b.view(n, CHUNK, H, -1), torch.matmul(x.float(), rows[fidx].transpose(1, 2))


def _fwd(st):
    q, v, case = st["q"], st["v"].float(), st["case"]
    T, H, dk = q.shape
    n, band, bmask, fidx, fmask = _bands(st)
    scale = 1.0 / math.sqrt(dk)
    sb, sf = _dots(q, st["k"].float(), n, band, fidx)
    sb = torch.where(bmask[:, :, None], sb * scale, -math.inf).view(n * CHUNK, H, -1)[:T]
    sf = torch.where(fmask[:, None], sf * scale, -math.inf)
    m = torch.maximum(sb.amax(-1), sf.amax(-1))
    sink = st["sink"].float() if st["sink"] is not None else torch.full((H,), -math.inf, device=q.device)
    m = torch.maximum(m, sink)
    eb, ef = torch.exp(sb - m[..., None]), torch.exp(sf - m[..., None])
    den = eb.sum(-1) + ef.sum(-1) + torch.exp(sink - m)
    num = torch.matmul(_padded(eb, n).view(n, CHUNK * H, -1), v[band]).view(n * CHUNK, H, -1)[:T]
    num = num + torch.matmul(ef, v[fidx])
    return (num / den[..., None]).to(q.dtype), m + torch.log(den)


def _bwd(st):
    q, k, v, dt = st["q"], st["k"].float(), st["v"].float(), st["q"].dtype
    T, H, dk = q.shape
    n, band, bmask, fidx, fmask = _bands(st)
    scale = 1.0 / math.sqrt(dk)
    lse, dout = st["lse"], st["dout"]
    delta = (dout.float() * st["out"].float()).sum(-1)
    sb, sf = _dots(q, k, n, band, fidx)
    pb = torch.where(bmask[:, :, None], torch.exp(sb * scale - _padded(lse, n).view(n, CHUNK, H, 1)), 0.0)
    pf = torch.where(fmask[:, None], torch.exp(sf * scale - lse[..., None]), 0.0)
    db, df = _dots(dout, v, n, band, fidx)
    db = (pb * (db - _padded(delta, n).view(n, CHUNK, H, 1)) * scale).view(n, CHUNK * H, -1)
    df = pf * (df - delta[..., None]) * scale
    pb = pb.view(n, CHUNK * H, -1)
    qp, dp = _padded(q, n).view(n, CHUNK * H, -1), _padded(dout, n).view(n, CHUNK * H, -1)
    dq = torch.matmul(db, k[band]).view(n * CHUNK, H, -1)[:T] + torch.matmul(df, k[fidx])
    dkey, dval = torch.zeros_like(k), torch.zeros_like(v)
    dkey.index_add_(0, band.reshape(-1), torch.matmul(db.transpose(1, 2), qp).flatten(0, 1))
    dval.index_add_(0, band.reshape(-1), torch.matmul(pb.transpose(1, 2), dp).flatten(0, 1))
    dkey.index_add_(0, fidx.reshape(-1), torch.matmul(df.transpose(1, 2), q.float()).flatten(0, 1))
    dval.index_add_(0, fidx.reshape(-1), torch.matmul(pf.transpose(1, 2), dout.float()).flatten(0, 1))
    got = [dq.to(dt), dkey.to(dt), dval.to(dt)]
    if st["sink"] is not None:
        got.append(-(torch.exp(st["sink"] - lse) * delta).sum(0))
    return got


def _append(st):
    case, page, cu = st["case"], st["case"]["page"], st["cu"].long()
    i = torch.arange(st["k"].shape[0], device=cu.device)
    s = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    pos = st["lens"][s] - cu[s + 1] + i
    pages, slots = st["table"][s, pos // page].long(), pos % page
    got = []
    for x, cache in ((st["k"], st["kc"]), (st["v"], st["vc"])):
        if x is not None:
            _write(cache, x.shape[1], page, pages, slots, x)
            got.append(_gather(cache, x.shape[1], page, pages, slots).to(torch.bfloat16))
    return got


def _positions(st):
    """Cached positions each query attends [S, N] and their mask."""
    case, lens = st["case"], st["lens"].long()[:, None]
    W, F = case["window"], case["first"]
    if not W:
        pos = torch.arange(st["maxlen"], device=lens.device)[None].expand(len(lens), -1)
        return pos, pos < lens
    x = torch.arange(min(W + F, st["maxlen"]), device=lens.device)[None]
    nf = torch.clamp(lens, max=F)
    pos = torch.where(x < nf, x, torch.maximum(nf, lens - W) + x - nf)
    mask = pos < lens
    return torch.where(mask, pos, 0), mask


def _decode(st):
    case, page, q = st["case"], st["case"]["page"], st["q"]
    pos, mask = _positions(st)
    pages, slots = torch.gather(st["table"].long(), 1, pos // page), pos % page
    k = _gather(st["kc"], case["dk"], page, pages, slots)
    v = k[..., :case["dv"]] if case["alias"] else _gather(st["vc"], case["dv"], page, pages, slots)
    s = torch.matmul(q.float(), k.transpose(1, 2)) / math.sqrt(case["dk"])
    s = torch.where(mask[:, None], s, -math.inf)
    m = s.amax(-1)
    sink = st["sink"].float() if st["sink"] is not None else torch.full_like(m, -math.inf)
    m = torch.maximum(m, sink)
    e = torch.exp(s - m[..., None])
    den = e.sum(-1) + torch.exp(sink - m)
    return [(torch.matmul(e, v) / den[..., None]).to(q.dtype), m + torch.log(den)]


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"fwd": _fwd, "bwd": _bwd, "append": _append, "decode": _decode}[op](st)
    from block_sparse_mqa_b200 import hs
    if op == "fwd":
        return hs.hs_swa_first_mqa_fwd(st["q"], st["k"], st["v"], st["cu"], st["maxlen"], case["window"],
                                       case["first"], st["sink"])
    if op == "bwd":
        g = hs.hs_swa_first_mqa_bwd(st["q"], st["k"], st["v"], st["cu"], st["maxlen"], case["window"],
                                    case["first"], st["out"], st["lse"], st["dout"], st["sink"])
        return [x for x in g if x is not None]
    if op == "append":
        hs.hs_kv4_append(st["k"], st["v"], st["kc"], st["vc"], st["table"], st["cu"], st["lens"], case["page"])
        return [hs.hs_kv4_read(cache, x.shape[1], st["table"], st["cu"], st["lens"], case["page"], x.shape[0])
                for x, cache in ((st["k"], st["kc"]), (st["v"], st["vc"])) if x is not None]
    return list(hs.hs_kv4_mqa_decode(st["q"], st["kc"], st["vc"], st["table"], st["lens"], st["maxlen"],
                                     case["page"], case["dv"], case["window"], case["first"], st["sink"]))


# ------------------------------------------------------------------ 64 bits
def _value64(codes, byte):
    """Codes [..., G, 16] and scales [..., G] -> float64 values: words, shifts and
    powers of two instead of bytes and halves."""
    word = codes.contiguous().view(torch.int32).long()
    e = torch.arange(8, device=codes.device)
    n = (word[..., None] >> (4 * (e // 2) + 16 * (e % 2))) & 15
    b = byte.long()
    ex, ma = b >> 3, b & 7
    scale = torch.where(ex > 0, ma + 8, ma).double() * torch.exp2((ex.clamp(min=1) - 18).double())
    return ((n.flatten(-2) - 8).double() * scale[..., None]).flatten(-2)


def _exact_attention(case, st, grad):
    """Forward or backward, a few hundred queries at a time over just their keys."""
    q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
    T, H, dk = q.shape
    scale, cu = dk ** -0.5, st["cu"].tolist()
    W, F = case["window"], case["first"]
    sink = st["sink"].double() if st["sink"] is not None else None
    out, lse = q.new_zeros(T, H, v.shape[1]), q.new_zeros(T, H)
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, b in zip(cu, cu[1:]):
        for c0 in range(a, b, 256):
            c1 = min(b, c0 + 256)
            w0 = max(a, c0 - W + 1)
            j = torch.cat((torch.arange(a, min(a + F, w0)), torch.arange(w0, c1))).to(q.device)
            t = torch.arange(c0, c1, device=q.device)[:, None]
            see = (j <= t) & ((j > t - W) | (j < a + F))
            s = torch.einsum("thd,jd->thj", q[c0:c1], k[j]) * scale
            if grad:
                p = torch.exp(s - st["lse"][c0:c1, :, None].double()) * see[:, None]
                do = st["dout"][c0:c1].double()
                delta = (do * st["out"][c0:c1].double()).sum(-1, keepdim=True)
                ds = p * (torch.einsum("thd,jd->thj", do, v[j]) - delta) * scale
                dq[c0:c1] = torch.einsum("thj,jd->thd", ds, k[j])
                dk_[j] += torch.einsum("thj,thd->jd", ds, q[c0:c1])
                dv_[j] += torch.einsum("thj,thd->jd", p, do)
                continue
            s = s.masked_fill(~see[:, None], -math.inf)
            l = torch.logsumexp(s, -1)
            lse[c0:c1] = l if sink is None else torch.logaddexp(l, sink.expand_as(l))
            out[c0:c1] = torch.einsum("thj,jd->thd", torch.exp(s - lse[c0:c1, :, None]), v[j])
    if not grad:
        return out, lse
    got = [dq, dk_, dv_]
    if sink is not None:
        delta = (st["dout"].double() * st["out"].double()).sum(-1)
        got.append(-(torch.exp(sink - st["lse"].double()) * delta).sum(0))
    return got


def _exact_append(st):
    got = []
    for x in (st["k"], st["v"]):
        if x is None:
            continue
        g = x.double().unflatten(-1, (-1, GROUP))
        r = g.abs().amax(-1) / 7
        # the smallest m * 2^e >= r with m in 8..15 (or below 8 at the least e, -17)
        e = torch.floor(torch.log2(r.clamp(min=1e-300))).clamp(min=-14) - 3
        scale = (torch.ceil(r / torch.exp2(e)) * torch.exp2(e)).clamp(max=61440.0)
        code = torch.where(scale[..., None] > 0, g / scale[..., None], torch.zeros_like(g)).round().clamp(-7, 7)
        got.append((code * scale[..., None]).flatten(-2))
    return got


def _exact_decode(case, st):
    page, outs, lses = case["page"], [], []
    W, F = case["window"], case["first"]
    for s, n in enumerate(st["lens"].tolist()):
        see = list(range(n)) if not W else list(range(min(F, n))) + list(range(max(min(F, n), n - W), n))
        pos = torch.tensor(see, device=st["q"].device)
        pg, sl = st["table"][s][pos // page].long(), pos % page

        def rows(cache, width):
            G = width // GROUP
            c = cache[:, :G * page * 16].view(-1, G, page, 16)[pg, :, sl]
            b = cache[:, G * page * 16:].view(len(cache), -1, page, 4)[pg, :, sl].flatten(-2)[:, :G]
            return _value64(c, b)

        k = rows(st["kc"], case["dk"])
        v = k[:, :case["dv"]] if case["alias"] else rows(st["vc"], case["dv"])
        x = st["q"][s].double() @ k.T * case["dk"] ** -0.5
        l = torch.logsumexp(x, -1)
        if st["sink"] is not None:
            l = torch.logaddexp(l, st["sink"].double())
        outs.append(torch.exp(x - l[:, None]) @ v)
        lses.append(l)
    return [torch.stack(outs), torch.stack(lses)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        return _exact_attention(case, st, case["op"] == "bwd")
    return _exact_append(st) if case["op"] == "append" else _exact_decode(case, st)
