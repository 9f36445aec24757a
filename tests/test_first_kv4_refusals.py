"""Host checks of the window attention with visible first tokens and of the
4-bit cache: refused before any CUDA call, so no GPU is needed."""

import ctypes

import pytest
import torch

from block_sparse_mqa_b200 import hs

INV, UNS, WSP = hs.HS_ERR_INVALID_ARG, hs.HS_ERR_UNSUPPORTED, hs.HS_ERR_WORKSPACE


def _call(fn, spec, kw):
    a = dict(spec)
    assert set(kw) <= set(a), kw
    a.update(kw)
    ptr = lambda x: ctypes.c_void_p(x) if x is not None else None
    types = getattr(hs.lib(), fn).argtypes
    st = getattr(hs.lib(), fn)(*[ptr(v) if t is ctypes.c_void_p else v for v, t in zip(a.values(), types)])
    assert st == hs.HS_OK or hs.lib().hs_last_error()
    return st


ATT = dict(q=256, qrs=64 * 576, qhs=576, k=256, krs=576, v=256, vrs=512, cu=256, nd=1, T=100, maxlen=100, H=64,
           dk=576, dv=512, dt=hs.HS_BF16, scale=0.0, window=16, first=2, sink=None)
FWD = dict(ATT, out=256, lse=256, stream=None)
BWD = dict(ATT, out=256, lse=256, dout=256, dq=256, dkey=256, dval=256, dsink=None, ws=256, wsb=1 << 40, stream=None)
COMMON = [(dict(window=0), INV), (dict(window=-3), INV), (dict(first=-1), INV), (dict(q=None), INV), (dict(k=None), INV),
          (dict(v=None), INV), (dict(cu=None), INV), (dict(T=-1), INV), (dict(nd=0), INV), (dict(maxlen=0), INV),
          (dict(H=0), UNS), (dict(H=129), UNS), (dict(dk=0), UNS), (dict(dk=2000), UNS), (dict(dv=0), UNS),
          (dict(dt=7), UNS), (dict(qhs=5), INV), (dict(qrs=576), INV), (dict(krs=5), INV), (dict(vrs=5), INV),
          (dict(scale=float("nan")), INV), (dict(out=None), INV), (dict(lse=None), INV)]


@pytest.mark.parametrize("kw,code", COMMON)
def test_window_first_forward_refuses(kw, code):
    assert _call("hs_swa_first_mqa_fwd", FWD, kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [(dict(dout=None), INV), (dict(dq=None), INV), (dict(dkey=None), INV),
                                              (dict(dval=None), INV), (dict(ws=None), WSP), (dict(wsb=1000), WSP),
                                              (dict(ws=258), INV)])
def test_window_first_backward_refuses(kw, code):
    assert _call("hs_swa_first_mqa_bwd", BWD, kw) == code


TABLE = dict(table=256, stride=4, width=4, pages=10, page=16)
APPEND = dict(k=256, krs=576, v=256, vrs=512, kc=256, vc=256, **TABLE, cu=256, lens=256, S=2, T=5, dk=576, dv=512,
              dt=hs.HS_BF16, stream=None)
READ = dict(cache=256, dim=576, **TABLE, cu=256, lens=256, S=2, T=5, out=256, ors=576, dt=hs.HS_BF16, stream=None)
DECODE = dict(q=256, qrs=64 * 576, qhs=576, kc=256, vc=256, **TABLE, lens=256, S=2, maxlen=64, H=64, dk=576, dv=512,
              dt=hs.HS_BF16, scale=0.0, window=0, first=0, sink=None, out=256, lse=256, ws=256, wsb=1 << 40, stream=None)
PAGED = [(dict(page=8), UNS), (dict(page=48), UNS), (dict(pages=-1), INV), (dict(S=-1), INV), (dict(table=None), INV),
         (dict(width=0), INV), (dict(stride=3), INV), (dict(dt=2), UNS), (dict(lens=None), INV)]


@pytest.mark.parametrize("kw,code", PAGED + [
    (dict(T=-1), INV), (dict(S=0), INV), (dict(cu=None), INV), (dict(dk=48), UNS), (dict(dk=0), UNS),
    (dict(dk=1056), UNS), (dict(dv=40), UNS), (dict(k=None), INV), (dict(kc=None), INV), (dict(v=None), INV),
    (dict(vc=None), INV), (dict(dv=0), INV), (dict(krs=100), INV), (dict(vrs=100), INV), (dict(kc=264), INV),
    (dict(vc=264), INV)])
def test_append_refuses(kw, code):
    assert _call("hs_kv4_append", APPEND, kw) == code


@pytest.mark.parametrize("kw,code", PAGED + [
    (dict(T=-1), INV), (dict(S=0), INV), (dict(cu=None), INV), (dict(dim=33), UNS), (dict(cache=None), INV),
    (dict(out=None), INV), (dict(ors=100), INV), (dict(cache=264), INV)])
def test_read_refuses(kw, code):
    assert _call("hs_kv4_read", READ, kw) == code


@pytest.mark.parametrize("kw,code", PAGED + [
    (dict(H=0), UNS), (dict(H=129), UNS), (dict(dk=48), UNS), (dict(dv=0), UNS), (dict(dv=1056), UNS),
    (dict(q=None), INV), (dict(kc=None), INV), (dict(out=None), INV), (dict(lse=None), INV), (dict(maxlen=0), INV),
    (dict(vc=None, dv=608), INV), (dict(qhs=100), INV), (dict(qrs=576), INV), (dict(scale=float("inf")), INV),
    (dict(window=-1), INV), (dict(first=-1), INV), (dict(first=3), INV), (dict(kc=264), INV), (dict(vc=264), INV),
    (dict(ws=None), WSP), (dict(wsb=16), WSP), (dict(ws=264), INV), (dict(S=2 ** 30), UNS),
    (dict(S=129, maxlen=2 ** 31 - 1), UNS), (dict(S=2 ** 20, maxlen=2 ** 31 - 1, window=2 ** 20, first=1), UNS)])
def test_decode_refuses(kw, code):
    assert _call("hs_kv4_mqa_decode", DECODE, kw) == code


def test_nothing_to_do_is_no_error():
    assert _call("hs_swa_first_mqa_fwd", FWD, dict(T=0, nd=0, maxlen=0)) == hs.HS_OK
    assert _call("hs_kv4_append", APPEND, dict(T=0, S=0)) == hs.HS_OK
    assert _call("hs_kv4_read", READ, dict(T=0, S=0)) == hs.HS_OK
    assert _call("hs_kv4_mqa_decode", DECODE, dict(S=0, maxlen=0, ws=None)) == hs.HS_OK


def test_backward_workspace_of_a_loose_bound():
    """A max_seqlen above the tokens there are asks for no more than the tokens do."""
    size = lambda maxlen, span: hs.workspace_size(hs.HS_OP_SWA_FIRST_MQA_BWD, 1000, 2, maxlen, 64, 576, 512,
                                                  torch.bfloat16, span)
    assert size(10 ** 6, 2000) == size(1000, 2000) > 2 ** 28
    assert size(10 ** 6, 40) == size(1000, 40) < size(10 ** 6, 2000)


def test_table_strides():
    """A table of one row has the stride it likes; rows that overlap are not taken for rows side by side."""
    lens = torch.zeros(3, dtype=torch.int32)
    stride = lambda table: hs._table_args(table, lens[:table.shape[0]], 5, 16)[1]
    one = torch.zeros((1, 4), dtype=torch.int32)
    assert stride(one) == 4 and stride(one[:, 1:]) >= 3
    assert stride(torch.zeros((3, 6), dtype=torch.int32)[:, :4]) == 6
    assert stride(one.expand(3, 4)) == 0
    assert _call("hs_kv4_mqa_decode", DECODE, dict(stride=0)) == INV


def test_page_bytes():
    assert hs.kv4_page_bytes(32, 16) == 16 * 20
    assert hs.kv4_page_bytes(512, 64) == 64 * (256 + 16)  # 4.25 bits an element
    assert hs.kv4_page_bytes(576, 128) == 128 * (288 + 20)
    for width, page in ((0, 16), (33, 16), (1056, 16), (64, 0), (64, 24), (64, 256)):
        with pytest.raises(ValueError):
            hs.kv4_page_bytes(width, page)


def test_binding_refuses_cpu_tensors():
    q, k, i = torch.zeros(4, 2, 32), torch.zeros(4, 32), torch.zeros(2, dtype=torch.int32)
    c = torch.zeros((3, 16 * 20), dtype=torch.uint8)
    with pytest.raises(ValueError):
        hs.hs_swa_first_mqa_fwd(q, k, k, i, 4, 2, 1)
    with pytest.raises(ValueError):
        hs.hs_kv4_append(k, None, c, None, i[:1, None], i, i[:1], 16)
    with pytest.raises(ValueError):
        hs.hs_kv4_mqa_decode(q, c, None, torch.zeros((4, 1), dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 4,
                             16, 32)


class _Launch(Exception):
    pass


@pytest.fixture
def recorded(monkeypatch):
    """The binding on CPU tensors up to the library call, whose arguments it raises."""
    def call(fn, index, *args):
        raise _Launch(args)

    monkeypatch.setattr(hs, "_same_device", lambda *ts: 0)
    monkeypatch.setattr(hs, "_call", call)


def _backward(workspace):
    q, k, lse = torch.zeros(8, 4, 32), torch.zeros(8, 32), torch.zeros(8, 4)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    return hs.hs_swa_first_mqa_bwd(q, k, k, cu, 8, 4, 1, q, lse, q, workspace=workspace)


def _decode(workspace, maxlen=40, window=0, first=0):
    cache, table = torch.zeros((4, 16 * 20), dtype=torch.uint8), torch.zeros((2, 3), dtype=torch.int32)
    return hs.hs_kv4_mqa_decode(torch.zeros(2, 4, 32), cache, None, table, torch.zeros(2, dtype=torch.int32), maxlen, 16,
                                32, window, first, workspace=workspace)


@pytest.mark.parametrize("call", [_backward, _decode])
def test_a_workspace_that_is_not_one_piece(recorded, call):
    """Its number of elements says nothing about the bytes behind its first one."""
    size = 1 << 20
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(size), torch.zeros(2 * size, dtype=torch.uint8)[::2],
               torch.zeros(8, 4).expand(1000, 8, 4)):
        with pytest.raises(ValueError, match="workspace"):
            call(ws)
    for ws, n in ((torch.zeros(size, dtype=torch.uint8), size), (torch.zeros(1000, 8), 32000)):
        with pytest.raises(_Launch) as e:
            call(ws)
        assert e.value.args[0][-2:] == (ws.data_ptr(), n)


@pytest.mark.parametrize("far", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1])
def test_sizes_past_32_bits_are_not_cut(recorded, far):
    """A window, first tokens or bound past a C int mean what the largest int means."""
    top = 2 ** 31 - 1
    q, k, lse = torch.zeros(8, 4, 32), torch.zeros(8, 32), torch.zeros(8, 4)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    with pytest.raises(_Launch) as e:
        hs.hs_swa_first_mqa_fwd(q, k, k, cu, far, far, far)
    with pytest.raises(_Launch) as f:
        hs.hs_swa_first_mqa_bwd(q, k, k, cu, far, far, far, q, lse, q)
    with pytest.raises(_Launch) as g:
        _decode(torch.zeros(1 << 20), far, far, far)
    for args, n in ((e.value.args[0], 3), (f.value.args[0], 3), (g.value.args[0], 3)):
        assert sum(a == top for a in args if isinstance(a, int)) == n
        assert not any(a == far for a in args if isinstance(a, int))
    for low in (-1, -2 ** 31 - 1, -2 ** 40):  # refused by the library, whatever bits they end in
        with pytest.raises(_Launch) as e:
            hs.hs_swa_first_mqa_fwd(q, k, k, cu, 8, low, 1)
        assert any(isinstance(a, int) and -2 ** 31 <= a < 0 for a in e.value.args[0])


@pytest.mark.parametrize("dk,dv,dt", [(576, 512, torch.float32), (96, 32, torch.bfloat16)])
def test_decode_workspace_of_the_largest_bound(dk, dv, dt):
    """A bound of the largest int asks for what one a little below it does."""
    size = lambda maxlen: hs.workspace_size(hs.HS_OP_KV4_MQA_DECODE, 2, 2, maxlen, 64, dk, dv, dt, 16)
    assert size(2 ** 31 - 1) == size(2 ** 31 - 5000) > size(64)


@pytest.mark.parametrize("kw,code", [(dict(dk=0), UNS), (dict(dt=7), UNS), (dict(window=0), INV), (dict(out=None), INV),
                                     (dict(dq=None), INV), (dict(scale=float("nan")), INV), (dict(krs=5), INV)])
def test_backward_of_no_tokens_refuses_first(kw, code):
    """The sink's gradient is cleared only by a call whose arguments are right."""
    assert _call("hs_swa_first_mqa_bwd", BWD, dict(T=0, nd=0, maxlen=0, sink=256, dsink=256, **kw)) == code


@pytest.mark.parametrize("H,dk,dv,dt", [(64, 576, 512, torch.bfloat16), (128, 576, 512, torch.bfloat16),
                                        (128, 1024, 1024, torch.float32), (1, 32, 32, torch.bfloat16)])
def test_decode_workspace_does_not_grow_with_the_batch(H, dk, dv, dt):
    """Partial results of as many pieces as fill the GPU, and 4 bytes a sequence."""
    for S in (1, 7, 100, 2000, 70001):
        for most in (1, 200, 10 ** 5):
            need = hs.workspace_size(hs.HS_OP_KV4_MQA_DECODE, S, S, most, H, dk, dv, dt, 64)
            assert need <= 148 * 2 * 64 * (8 + 4 * dv) + 4 * S + 16, (S, most, need)
    assert _call("hs_kv4_mqa_decode", DECODE, dict(S=0, maxlen=0, ws=None)) == hs.HS_OK
