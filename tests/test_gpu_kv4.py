"""The 4-bit paged cache: rows written and read exactly as oracle/kv4.py says,
decode against a float64 form over the cached values (bounds: tests/attn64.py),
and the calls together."""

import numpy as np
import pytest
import torch

import oracle.kv4 as K4
from block_sparse_mqa_b200 import hs
from tests import attn64 as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _i32(x):
    return torch.tensor(x, device=DEV, dtype=torch.int32)


def _table(lens, page, seed=0, spare=3):
    """A block table with shuffled pages (-1 where no page is needed) and the pool's size."""
    need = [-(-n // page) for n in lens]
    perm = np.random.default_rng(seed).permutation(sum(need) + spare)
    t, at = np.full((len(lens), max([1] + need)), -1, np.int32), 0
    for i, n in enumerate(need):
        t[i, :n] = perm[at:at + n]
        at += n
    return torch.tensor(t, device=DEV), len(perm)


def _cu(lens):
    return _i32(np.cumsum([0] + list(lens)))


def _values(x):
    """float64 values of quantised rows (oracle)."""
    return K4.values(*K4.quantise(x.double().cpu().numpy()))


# ------------------------------------------------------------------ append and read
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv,page", [(32, 0, 16), (96, 64, 32), (160, 128, 64), (576, 512, 128), (1024, 32, 16)])
def test_append_then_read(dk, dv, page, dtype):
    old, new = [0, 5, 15, 0, 16, 40], [3, 1, 2, 0, 16, 30]
    total = [a + b for a, b in zip(old, new)]
    table, pool = _table(total, page)
    g = torch.Generator(device=DEV)
    g.manual_seed(dk)
    n = sum(new)
    k = (torch.randn((n, dk), generator=g, device=DEV) * torch.exp2(torch.randint(-9, 9, (n, 1), device=DEV))).to(dtype)
    v = torch.randn((n, dv), generator=g, device=DEV).to(dtype) if dv else None
    kc = hs.kv4_cache(pool, dk, page)
    vc = hs.kv4_cache(pool, dv, page) if dv else None
    kc.fill_(0xEE)
    hs.hs_kv4_append(k, v, kc, vc, table, _cu(new), _i32(total), page)
    hs.poll_status()
    # the pages, byte by byte
    want = np.full(kc.shape, 0xEE, np.uint8)
    codes, byte = K4.quantise(k.double().cpu().numpy())
    tab, row = table.cpu().numpy(), 0
    for s, (a, b) in enumerate(zip(old, new)):
        for pos in range(a, a + b):
            K4.pack_row(want[tab[s, pos // page]], dk, page, pos % page, codes[row], byte[row])
            row += 1
    assert np.array_equal(kc.cpu().numpy(), want)
    for x, c in ((k, kc), (v, vc)):
        if x is None:
            continue
        for out_dtype in (F32, BF16):
            got = hs.hs_kv4_read(c, x.shape[1], table, _cu(new), _i32(total), page, n, dtype=out_dtype)
            assert np.array_equal(got.double().cpu().numpy(), _values(x))
    hs.poll_status()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_append_special_values(dtype):
    """Zero, subnormal, tiny, huge and non-finite groups, and ties between codes."""
    rows = torch.zeros((10, 64), device=DEV)
    rows[1, :4] = torch.tensor([1e-40, -1e-40, 1e-38, 0])
    rows[2, :3] = torch.tensor([2.0 ** -17 * 7, 2.0 ** -18, -2.0 ** -18])
    rows[3, :3] = torch.tensor([430080.0, 30720.0, -1e5])
    rows[4, :2] = torch.tensor([3e38, -1e30])
    rows[5, 40], rows[6, 3], rows[7, 33] = float("nan"), float("inf"), float("-inf")
    rows[8, :8] = torch.tensor([7, 0.5, 1.5, 2.5, -0.5, -1.5, 6.5, -6.5])  # scale 1: ties to even
    rows[9, :32] = torch.linspace(-3.5, 3.5, 32, device=DEV)
    x = rows.to(dtype)
    table, pool = _table([10], 16)
    kc = hs.kv4_cache(pool, 64, 16)
    hs.hs_kv4_append(x, None, kc, None, table, _cu([10]), _i32([10]), 16)
    got = hs.hs_kv4_read(kc, 64, table, _cu([10]), _i32([10]), 16, 10, dtype=F32).double().cpu().numpy()
    hs.poll_status()
    want = _values(x)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isnan(want[5, 32:]).all() and not np.isnan(want[5, :32]).any()


def test_append_next_to_code_and_scale_borders_fp32():
    """fp32 values one step around every border between two codes and two scales."""
    r = np.random.default_rng(1)
    x = np.zeros((400, 32), np.float32)
    for i in range(400):
        m, e = r.integers(8, 16), int(r.integers(-6, 6))
        s = float(m) * 2.0 ** e
        x[i, 0] = np.nextafter(np.float32(7 * s), np.float32(r.choice([0, 1e9]))) if i % 2 else 7 * s
        mid = (r.integers(0, 7, 31) + 0.5) * s
        x[i, 1:] = np.nextafter(mid.astype(np.float32), np.float32(r.choice([0, 1e9]))) * r.choice([-1, 1], 31)
    t = torch.tensor(x, device=DEV)
    table, pool = _table([400], 64)
    kc = hs.kv4_cache(pool, 32, 64)
    hs.hs_kv4_append(t, None, kc, None, table, _cu([400]), _i32([400]), 64)
    got = hs.hs_kv4_read(kc, 32, table, _cu([400]), _i32([400]), 64, 400, dtype=F32)
    assert np.array_equal(got.double().cpu().numpy(), _values(t))


def test_strided_rows_padding_rows_and_one_token():
    page, new = 16, [2, 0, 5]
    table, pool = _table([10, 4, 21], page)
    for pad, off in ((8, 8), (5, 1)):
        k = torch.randn((12, 96 + pad), device=DEV, dtype=BF16)[:, off:off + 96]  # 7 rows, 5 of padding
        kc = hs.kv4_cache(pool, 96, page)
        hs.hs_kv4_append(k, None, kc, None, table, _cu(new), _i32([10, 4, 21]), page)
        out = torch.full((12, 96 + pad), 9.0, device=DEV, dtype=BF16)[:, off:off + 96]
        hs.hs_kv4_read(kc, 96, table, _cu(new), _i32([10, 4, 21]), page, 12, out=out)
        hs.poll_status()
        assert np.array_equal(out[:7].double().cpu().numpy(), _values(k[:7]))
        assert bool((out[7:] == 9).all())
    one = torch.randn((1, 96), device=DEV)
    hs.hs_kv4_append(one, None, kc, None, table[1:2], _cu([1]), _i32([4]), page)
    got = hs.hs_kv4_read(kc, 96, table[1:2], _cu([1]), _i32([4]), page, 1, dtype=F32)
    assert np.array_equal(got.double().cpu().numpy(), _values(one))


def test_bad_pages_and_lengths_are_reported_and_skipped():
    page = 16
    k = torch.randn((4, 32), device=DEV)
    base = hs.kv4_cache(5, 32, page)
    for table, cu, lens, code in (
            ([[7]], [0, 4], [4], hs.HS_ERR_INVALID_INDEX),      # no such page
            ([[-1]], [0, 4], [4], hs.HS_ERR_INVALID_INDEX),
            ([[1]], [0, 4], [18], hs.HS_ERR_INVALID_INDEX),     # rows 14..17: 16 and 17 past the table
            ([[1]], [0, 4], [3], hs.HS_ERR_INVALID_ARG),        # more new rows than rows
            ([[1], [2]], [0, 5, 4], [5, 4], hs.HS_ERR_INVALID_ARG)):  # cu_seqlens goes down
        kc = base.clone()
        hs.hs_kv4_append(k, None, kc, None, _i32(table), _i32(cu), _i32(lens), page)
        with pytest.raises(hs.HSError) as e:
            hs.poll_status()
        assert e.value.status == code
        assert not kc[0].any() and not kc[3:].any()  # nothing outside the valid pages
        out = torch.full((4, 32), 9.0, device=DEV)
        hs.hs_kv4_read(kc, 32, _i32(table), _i32(cu), _i32(lens), page, 4, out=out)
        with pytest.raises(hs.HSError):
            hs.poll_status()
        assert bool((out[2:] == 9).all())


# ------------------------------------------------------------------ decode
def _cache(lens, width, page, seed, table=None, pool=None):
    """A plane whose sequences hold random rows; returns it with the rows' values [S][len, width]."""
    if table is None:
        table, pool = _table(lens, page, seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((max(1, sum(lens)), width), generator=g, device=DEV).to(BF16)
    c = hs.kv4_cache(pool, width, page)
    c.fill_(0xFF)  # pages nobody wrote read as NaN
    hs.hs_kv4_append(x, None, c, None, table, _cu(lens), _i32(lens), page)
    val = hs.hs_kv4_read(c, width, table, _cu(lens), _i32(lens), page, sum(lens), dtype=F32)
    return table, pool, c, list(val.split(list(lens)))


def _positions(n, window, first):
    return torch.tensor(K4.positions(n, window, first), device=DEV, dtype=torch.long)


def _decode(lens, H, dk, dv, page, window=0, first=0, dtype=BF16, alias=False, sink=True, seed=0, max_seqlen=None,
            path=None):
    table, pool, kc, kv = _cache(lens, dk, page, seed)
    vc, vv = (None, [x[:, :dv] for x in kv]) if alias else _cache(lens, dv, page, seed + 1, table, pool)[2:]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 2)
    q = torch.randn((len(lens), H, dk), generator=g, device=DEV).to(dtype)
    sk = torch.randn(H, generator=g, device=DEV) if sink else None
    if window:  # pages that no key needs may be missing
        for s, n in enumerate(lens):
            live = set((_positions(n, window, first) // page).tolist())
            for e in range(table.shape[1]):
                if e not in live:
                    table[s, e] = -5
    out, lse = hs.hs_kv4_mqa_decode(q, kc, vc, table, _i32(lens), max_seqlen or max(1, max(lens)), page, dv, window,
                                    first, sk)
    hs.poll_status()
    if path is not None:
        assert hs.last_path() == path
    _check_decode(q, kv, vv, lens, window, first, sk, out, lse, dtype)
    return out, lse


def _check_decode(q, kv, vv, lens, window, first, sk, out, lse, dtype):
    for s, n in enumerate(lens):
        if n == 0:
            assert not out[s].any()
            assert torch.equal(lse[s], sk if sk is not None else torch.full_like(lse[s], -torch.inf))
            continue
        pos = _positions(n, window, first)
        mask = torch.ones((1, len(pos)), dtype=torch.bool, device=DEV)
        ref, rl, bo, bl = A.forward(q[s:s + 1], kv[s][pos], vv[s][pos], mask, sk, q.shape[2] ** -0.5, dtype)
        A.check(out[s:s + 1], ref, bo, "out of sequence %d" % s)
        A.check(lse[s:s + 1], rl, bl, "lse of sequence %d" % s)


LENS = [1, 0, 2, 17, 128, 129, 300, 64, 1000, 5]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("alias", [False, True])
def test_decode_mla_shape(page, alias):
    _decode(LENS, 64, 576, 512, page, alias=alias, seed=page)


@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (7, 3), (128, 4), (124, 4), (300, 200), (5000, 9)])
def test_decode_window_and_first_tokens(window, first):
    _decode(LENS, 64, 576, 512, 16, window=window, first=first, alias=True, sink=first != 3, seed=3)


@pytest.mark.parametrize("H", [1, 7, 16, 63, 65, 128])
def test_decode_heads(H):
    _decode([40, 0, 333], H, 192, 128, 32, seed=4)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 512), (512, 512), (576, 448), (320, 256)])
def test_decode_widths(dk, dv):
    _decode([200, 131], 64, dk, dv, 64, seed=5)


@pytest.mark.parametrize("dk,dv,dtype", [(64, 64, F32), (576, 512, F32), (32, 32, BF16), (96, 160, BF16),
                                         (1024, 1024, F32), (608, 1024, BF16)])
def test_decode_other_shapes_and_fp32(dk, dv, dtype):
    for window, first in ((0, 0), (33, 2)):
        _decode([70, 1, 0, 150], 5, dk, dv, 16, window, first, dtype, seed=6)


@pytest.mark.parametrize("lens", [[1], [127], [20000], [3] * 700, [9000, 1, 1, 1, 8000] + [0] * 300 + [129]])
def test_decode_splits(lens):
    """One sequence over the whole GPU, many short ones, ragged and empty ones."""
    _decode(lens, 64, 192, 128, 64, seed=7)


def test_decode_max_seqlen_is_only_a_bound():
    a = _decode([300, 77], 64, 192, 128, 32, seed=8)
    b = _decode([300, 77], 64, 192, 128, 32, seed=8, max_seqlen=100000)
    # another split of the keys: within both bounds of the same values
    assert (a[0].float() - b[0].float()).abs().max() <= 0.1 and (a[1] - b[1]).abs().max() <= 1e-4


def test_decode_shared_pages():
    """Two sequences that share their first pages, and one table row used twice."""
    page, lens = 16, [64, 70]
    table, pool, kc, kv = _cache([64, 80], 192, page, 9)
    table[1, :4] = table[0, :4]
    kv1 = torch.cat((kv[0], kv[1][64:70]))
    q = torch.randn((3, 64, 192), device=DEV).to(BF16)
    t = torch.stack((table[0], table[1], table[0]))
    out, lse = hs.hs_kv4_mqa_decode(q, kc, None, t, _i32(lens + [64]), 80, page, 128)
    hs.poll_status()
    rows = [kv[0], kv1, kv[0]]
    _check_decode(q, rows, [x[:, :128] for x in rows], lens + [64], 0, 0, None, out, lse, BF16)


@pytest.mark.parametrize("dk,H,path", [(64, 16, hs.HS_PATH_TCGEN05), (96, 2, hs.HS_PATH_SIMT)])
def test_more_sequences_than_a_grid_dimension(dk, H, path):
    """70001 sequences, each one of five over shared pages; then a token appended to
    every one (pages of their own) and read back."""
    lens, S, page = [1, 40, 0, 16, 130], 70001, 16
    table, pool, kc, kv = _cache(lens, dk, page, 30)
    of = torch.arange(S, device=DEV) % 5
    q = torch.randn((5, H, dk), device=DEV).to(BF16)
    out, lse = hs.hs_kv4_mqa_decode(q[of], kc, None, table[of].contiguous(), _i32(lens)[of].contiguous(), 130, page, 64)
    assert hs.last_path() == path
    hs.poll_status()
    for s, n in enumerate(lens):
        if n == 0:
            assert not out[s::5].any() and bool((lse[s::5] == -torch.inf).all())
            continue
        mask = torch.ones((1, n), dtype=torch.bool, device=DEV)
        ref, rl, bo, bl = A.forward(q[s:s + 1], kv[s], kv[s][:, :64], mask, None, dk ** -0.5, BF16)
        A.check(out[s::5], ref.expand(out[s::5].shape), bo.expand(out[s::5].shape), "out")
        A.check(lse[s::5], rl.expand(lse[s::5].shape), bl.expand(lse[s::5].shape), "lse")
    x = torch.randn((S, dk), device=DEV).to(BF16)
    cache, own = hs.kv4_cache(S, dk, page), torch.arange(S, device=DEV, dtype=torch.int32)[:, None]
    cu, ones = torch.arange(S + 1, device=DEV, dtype=torch.int32), torch.ones(S, device=DEV, dtype=torch.int32)
    hs.hs_kv4_append(x, None, cache, None, own, cu, ones, page)
    got = hs.hs_kv4_read(cache, dk, own, cu, ones, page, S)
    hs.poll_status()
    some = slice(0, S, 997)
    assert torch.equal(got[some].double().cpu(), torch.tensor(_values(x[some])))


def test_decode_strided_and_unaligned_queries():
    lens, page = [90, 33], 32
    table, pool, kc, kv = _cache(lens, 192, page, 10)
    for off, pad in ((8, 8), (1, 3)):
        q = torch.randn((2, 66, 192 + pad), device=DEV, dtype=BF16)[:, 1:65, off:off + 192]
        out, lse = hs.hs_kv4_mqa_decode(q, kc, None, table, _i32(lens), 90, page, 128)
        hs.poll_status()
        _check_decode(q, kv, [x[:, :128] for x in kv], lens, 0, 0, None, out, lse, BF16)


def test_decode_nan_rows_outside_the_key_set():
    """The unused part of a page, and keys between the first tokens and the window, are NaN."""
    page, n, window, first = 64, 200, 30, 3
    table, pool, kc, kv = _cache([n], 576, page, 11)
    bad = torch.full((1, 576), float("nan"), device=DEV)
    for pos in (3, 50, 169):  # neighbours of the visible positions, and one between
        hs.hs_kv4_append(bad, None, kc, None, table, _cu([1]), _i32([pos + 1]), page)
    q = torch.randn((1, 64, 576), device=DEV).to(BF16)
    out, lse = hs.hs_kv4_mqa_decode(q, kc, None, table, _i32([n]), n, page, 512, window, first)
    hs.poll_status()
    _check_decode(q, kv, [x[:, :512] for x in kv], [n], window, first, None, out, lse, BF16)
    full, _ = hs.hs_kv4_mqa_decode(q, kc, None, table, _i32([n]), n, page, 512)
    assert bool(full.isnan().all())  # a NaN that is attended is not hidden


def test_decode_bad_lengths_and_pages_are_reported():
    page = 16
    table, pool, kc, kv = _cache([40, 20], 64, page, 12)
    q = torch.randn((2, 64, 64), device=DEV).to(BF16)
    bad = table.clone()
    bad[0, 1] = pool
    for t, lens, most, code in ((table, [40, 21], 40, None), (table, [41, 20], 40, hs.HS_ERR_INVALID_ARG),
                                (table, [-1, 20], 40, hs.HS_ERR_INVALID_ARG),
                                (bad, [40, 20], 40, hs.HS_ERR_INVALID_INDEX),
                                (table, [40, 60], 60, hs.HS_ERR_INVALID_INDEX)):  # past the table
        out, lse = hs.hs_kv4_mqa_decode(q, kc, None, t, _i32(lens), most, page, 64)
        if code is None:
            hs.poll_status()
            continue
        with pytest.raises(hs.HSError) as e:
            hs.poll_status()
        assert e.value.status == code
        if code == hs.HS_ERR_INVALID_ARG:  # treated as an empty sequence
            assert not out[0].any() and bool((lse[0] == -torch.inf).all())
            _check_decode(q[1:], kv[1:], kv[1:], [20], 0, 0, None, out[1:], lse[1:], BF16)


@pytest.mark.parametrize("dk,path", [(64, hs.HS_PATH_TCGEN05), (96, hs.HS_PATH_SIMT)])
def test_decode_lengths_at_the_end_of_int(dk, path):
    """The largest int as bound, and as a length: reported, and no key of it is looked for."""
    page, lens = 16, [40, 2 ** 31 - 1, 20, 2 ** 31 - 4095]
    table, pool, kc, kv = _cache([40, 1, 20, 1], dk, page, 31)
    q = torch.randn((4, 64, dk), device=DEV).to(BF16)
    for window, first in ((0, 0), (10, 2)):
        out, lse = hs.hs_kv4_mqa_decode(q, kc, None, table, _i32(lens), 2 ** 31 - 1, page, 64, window, first)
        assert hs.last_path() == path
        with pytest.raises(hs.HSError) as e:
            hs.poll_status()
        assert e.value.status == hs.HS_ERR_INVALID_ARG
        n, val = [40, 0, 20, 0], [kv[0], kv[0][:0], kv[2], kv[0][:0]]
        _check_decode(q, val, [x[:, :64] for x in val], n, window, first, None, out, lse, BF16)


def test_decode_streams_and_graphs_with_growing_sequences():
    """A captured step (append one token to each sequence, attend) replayed while
    the lengths move on the device; two graphs and an eager call, each its own workspace."""
    page, S, width, dv, start = 16, 3, 192, 128, [14, 31, 100]
    cap = [n + 8 for n in start]
    table, pool = _table(cap, page, 13)
    g = torch.Generator(device=DEV)
    g.manual_seed(13)
    new = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF16)
    x0 = new(sum(start), width)
    kc = hs.kv4_cache(pool, width, page)
    hs.hs_kv4_append(x0, None, kc, None, table, _cu(start), _i32(start), page)
    rows = list(x0.split(start))
    lens, k1, q = _i32(start), new(S, width), new(S, 64, width)
    cu1, most = _cu([1] * S), max(cap)

    def step():
        lens.add_(1)
        hs.hs_kv4_append(k1, None, kc, None, table, cu1, lens, page)
        return hs.hs_kv4_mqa_decode(q, kc, None, table, lens, most, page, dv, 40, 2)

    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            held = step()
        graphs.append((gr, held))
    side = torch.cuda.Stream()
    for i in range(6):
        k1.copy_(new(S, width))
        q.copy_(new(S, 64, width))
        rows = [torch.cat((r, k1[s:s + 1])) for s, r in enumerate(rows)]
        if i % 3 == 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                out, lse = step()
            torch.cuda.current_stream().wait_stream(side)
        else:
            graphs[i % 3][0].replay()
            out, lse = graphs[i % 3][1]
        hs.poll_status()
        val = [torch.tensor(_values(r), device=DEV) for r in rows]
        n = [len(r) for r in rows]
        assert lens.tolist() == n
        _check_decode(q, val, [x[:, :dv] for x in val], n, 40, 2, None, out, lse, BF16)


def test_two_calls_at_once():
    lens, page = [2000, 700, 1], 64
    table, pool, kc, kv = _cache(lens, 576, page, 14)
    q = [torch.randn((3, 64, 576), device=DEV).to(BF16) for _ in range(4)]
    want = [hs.hs_kv4_mqa_decode(x, kc, None, table, _i32(lens), 2000, page, 512) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    got, sl = [], _i32(lens)
    torch.cuda.synchronize()
    for x, s in zip(q, streams):
        with torch.cuda.stream(s):
            got.append([hs.hs_kv4_mqa_decode(x, kc, None, table, sl, 2000, page, 512) for _ in range(3)][-1])
    torch.cuda.synchronize()
    hs.poll_status()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_far_pages_pass_32_bit_offsets():
    """Pages beyond 4 GiB of the cache."""
    page, width = 128, 576
    pool = (4 << 30) // hs.kv4_page_bytes(width, page) + 40
    kc = torch.empty((pool, hs.kv4_page_bytes(width, page)), dtype=torch.uint8, device=DEV)
    table = _i32([[pool - 1, 3, pool - 20]])
    x = torch.randn((300, width), device=DEV).to(BF16)
    hs.hs_kv4_append(x, None, kc, None, table, _cu([300]), _i32([300]), page)
    val = hs.hs_kv4_read(kc, width, table, _cu([300]), _i32([300]), page, 300, dtype=F32)
    assert np.array_equal(val.double().cpu().numpy(), _values(x))
    q = torch.randn((1, 64, width), device=DEV).to(BF16)
    out, lse = hs.hs_kv4_mqa_decode(q, kc, None, table, _i32([300]), 300, page, 512)
    hs.poll_status()
    _check_decode(q, [val], [val[:, :512]], [300], 0, 0, None, out, lse, BF16)


def test_prompt_then_tokens_as_a_model_would():
    """A prompt runs through the window attention with visible first tokens, its
    keys enter the cache, and the next tokens are decoded from it: each agrees
    with the forward over the cached values."""
    page, W, F, docs, dk, dv = 32, 48, 4, [130, 77], 576, 512
    T = sum(docs)
    g = torch.Generator(device=DEV)
    g.manual_seed(15)
    new = lambda *s: torch.randn(s, generator=g, device=DEV).to(BF16)
    q, k, sink = new(T, 64, dk), new(T, dk), torch.randn(64, generator=g, device=DEV)
    cap = [n + 5 for n in docs]
    table, pool = _table(cap, page, 15)
    kc = hs.kv4_cache(pool, dk, page)
    hs.hs_kv4_append(k, None, kc, None, table, _cu(docs), _i32(docs), page)
    kq = hs.hs_kv4_read(kc, dk, table, _cu(docs), _i32(docs), page, T)
    hs.hs_swa_first_mqa_fwd(q, kq, kq[:, :dv], _cu(docs), max(docs), W, F, sink)
    n = list(docs)
    for _ in range(5):
        n = [x + 1 for x in n]
        hs.hs_kv4_append(new(2, dk), None, kc, None, table, _cu([1, 1]), _i32(n), page)
        q1 = new(2, 64, dk)
        out, lse = hs.hs_kv4_mqa_decode(q1, kc, None, table, _i32(n), max(cap), page, dv, W, F, sink)
        kq = hs.hs_kv4_read(kc, dk, table, _cu(n), _i32(n), page, sum(n))
        qq = torch.zeros((sum(n), 64, dk), device=DEV, dtype=BF16)
        last = torch.tensor(np.cumsum(n) - 1, device=DEV)
        qq[last] = q1
        fo, fl = hs.hs_swa_first_mqa_fwd(qq, kq, kq[:, :dv], _cu(n), max(n), W, F, sink)
        hs.poll_status()
        # each side is two bf16 roundings from the same value, of size |v|
        size = kq.float().abs().max()
        assert (out.float() - fo[last].float()).abs().max() <= 4 * 2.0 ** -8 * size
        assert (lse - fl[last]).abs().max() <= 1e-4
