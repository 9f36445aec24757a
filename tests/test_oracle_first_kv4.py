"""Pins, without a GPU, of the definitions behind the window attention with
visible first tokens and the 4-bit cache: against loops, autograd, finite
differences, other functions of the oracle, and closed forms."""

import numpy as np
import pytest
import torch

import oracle.backward as OB
import oracle.hysparse as O
import oracle.kv4 as K4
import oracle.loops as L

RNG = np.random.default_rng


def _case(docs, H=2, dk=5, dv=3, seed=0):
    r, T = RNG(seed), sum(docs)
    return (r.standard_normal((T, H, dk)), r.standard_normal((T, dk)), r.standard_normal((T, dv)),
            r.standard_normal(H), list(np.cumsum([0] + docs)))


def _mask(cu, window, first):
    T = cu[-1]
    m = [[False] * T for _ in range(T)]
    for bos, eos in zip(cu, cu[1:]):
        for t in range(bos, eos):
            for j in range(bos, t + 1):
                m[t][j] = t - j < window or j - bos < first
    return m


@pytest.mark.parametrize("window,first", [(1, 0), (1, 1), (3, 2), (4, 9), (50, 1)])
def test_first_window_forward_is_the_masked_loop(window, first):
    q, k, v, sink, cu = _case([7, 1, 12])
    ref = O.swa_first_mqa_fwd(q, k, v, cu, window, first, sink)
    out, lse = L.masked_attention(q.tolist(), k.tolist(), v.tolist(), _mask(cu, window, first),
                                  sink.tolist(), 5 ** -0.5)
    np.testing.assert_allclose(ref["out"], out, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(ref["lse"], lse, rtol=1e-12, atol=1e-13)


def test_no_first_tokens_is_the_window_and_all_of_them_dense():
    q, k, v, sink, cu = _case([9, 14])
    a, b = O.swa_first_mqa_fwd(q, k, v, cu, 4, 0, sink), O.swa_mqa_fwd(q, k, v, cu, 4, sink)
    assert np.array_equal(a["out"], b["out"]) and np.array_equal(a["lse"], b["lse"])
    a, b = O.swa_first_mqa_fwd(q, k, v, cu, 2, 14, sink), O.dense_causal_fwd(q, k, v, cu, sink)
    assert np.array_equal(a["out"], b["out"]) and np.array_equal(a["lse"], b["lse"])


@pytest.mark.parametrize("window,first", [(1, 1), (3, 2), (5, 20)])
def test_first_window_backward_against_autograd_and_differences(window, first):
    q, k, v, sink, cu = _case([8, 11], seed=1)
    dout = RNG(5).standard_normal((19, 2, 3))
    got = OB.swa_first_mqa_bwd(q, k, v, dout, cu, window, first, sink)
    t = [torch.tensor(x, dtype=torch.float64, requires_grad=True) for x in (q, k, v, sink)]
    s = torch.einsum("thd,jd->thj", t[0], t[1]) * 5 ** -0.5
    s = s.masked_fill(~torch.tensor(_mask(cu, window, first))[:, None], -torch.inf)
    p = torch.softmax(torch.cat((s, t[3].view(1, 2, 1).expand(19, 2, 1)), -1), -1)[..., :-1]
    (torch.einsum("thj,jd->thd", p, t[2]) * torch.tensor(dout)).sum().backward()
    for x, name in zip(t, ("dq", "dk", "dv", "dsink")):
        np.testing.assert_allclose(got[name], x.grad.numpy(), rtol=1e-10, atol=1e-12)

    def loss(k_):
        return float((O.swa_first_mqa_fwd(q, k_, v, cu, window, first, sink)["out"] * dout).sum())

    for j, d in ((0, 0), (8, 2), (18, 4)):  # a first token of each document, a last one
        e = np.zeros_like(k)
        e[j, d] = 1e-5
        assert abs((loss(k + e) - loss(k - e)) / 2e-5 - got["dk"][j, d]) < 1e-7


# ------------------------------------------------------------------ 4-bit format
def test_every_scale_byte_is_the_half_with_its_upper_bits():
    b = np.arange(248, dtype=np.uint16)
    halves = (b << 7).astype(np.uint16).view(np.float16).astype(np.float64)
    assert np.array_equal(halves, [K4.byte_value(int(x)) for x in b])
    assert np.isnan((np.uint16(255) << np.uint16(7)).astype(np.uint16).view(np.float16))


def test_scale_is_the_smallest_that_covers():
    r = RNG(2)
    amax = np.concatenate((r.standard_normal(300) ** 2, 2.0 ** r.uniform(-30, 25, 300), [0.0, 7.0, 1e9]))
    for a in amax:
        byte, s = K4.scale_of(a)
        assert s == K4.byte_value(byte)
        if byte == 247:
            assert s == 61440.0
            continue
        assert 7 * s >= a and (byte == 0 or 7 * K4.byte_value(byte - 1) < a)


def test_quantisation_error_and_exactness_in_bf16():
    x = RNG(3).standard_normal((40, 96)) * np.exp(RNG(4).uniform(-6, 6, (40, 1)))
    codes, byte = K4.quantise(x)
    val = K4.values(codes, byte)
    step = np.repeat(np.asarray([[K4.byte_value(int(b)) for b in row] for row in byte]), 32, axis=1)
    assert np.all(np.abs(val - x) <= step / 2)  # half a code
    assert np.all(step <= np.repeat(np.abs(x).reshape(40, 3, 32).max(-1) / 7 * 1.125, 32, axis=1))
    t = torch.tensor(val)
    assert torch.equal(t, t.to(torch.bfloat16).double())


def test_special_groups():
    x = np.zeros((4, 32))
    x[1, 3], x[2, 4], x[3, :2] = np.nan, np.inf, (1e6, -1.0)
    codes, byte = K4.quantise(x)
    assert byte[:, 0].tolist() == [0, 255, 255, 247]
    val = K4.values(codes, byte)
    assert np.all(val[0] == 0) and np.all(np.isnan(val[1:3]))
    assert val[3, 0] == 430080.0 and val[3, 1] == 0.0


@pytest.mark.parametrize("width,page", [(32, 16), (96, 16), (128, 32), (576, 64)])
def test_pages_hold_rows_without_overlap(width, page):
    r = RNG(6)
    rows = r.standard_normal((page, width))
    codes, byte = K4.quantise(rows)
    buf = np.full(K4.page_bytes(width, page), 0xEE, np.uint8)
    for s in r.permutation(page):
        K4.pack_row(buf, width, page, s, codes[s], byte[s])
    for s in range(page):
        assert np.array_equal(K4.unpack_row(buf, width, page, s), K4.values(codes[s:s + 1], byte[s:s + 1])[0])
    assert int((buf == 0xEE).sum()) >= page * (4 * -(-width // 128) - width // 32)  # the unused scale bytes


def test_decode_is_the_last_row_of_the_forward():
    q, k, v, sink, cu = _case([23], dk=6, dv=4)
    for window, first in ((0, 0), (5, 0), (5, 3), (2, 40)):
        out, lse = K4.decode(q[-1:], [k], [v], window, first, sink)
        ref = O.swa_first_mqa_fwd(q, k, v, cu, window or 23, first, sink, rows=[22])
        np.testing.assert_allclose(out, ref["out"], rtol=1e-13)
        np.testing.assert_allclose(lse, ref["lse"], rtol=1e-13)
    out, lse = K4.decode(q[-1:], [k[:0]], [v[:0]], 0, 0, sink)
    assert not out.any() and np.array_equal(lse[0], sink)
