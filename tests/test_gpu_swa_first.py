"""hs_swa_first_mqa_fwd / _bwd against a dense-mask form in float64
(tests/attn64.py, which also gives the error bounds), and against the oracle."""

import ctypes

import numpy as np
import pytest
import torch

import oracle.hysparse as O
from block_sparse_mqa_b200 import hs, synth
from tests import attn64 as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _inputs(docs, H, dk, dv, dtype, seed):
    inp = synth.make_inputs(sum(docs), H, dk, dv, dtype=dtype, seed=seed, device=DEV, doc_lengths=docs)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 77)
    dout = torch.randn((sum(docs), H, dv), generator=g, device=DEV).to(dtype)
    return inp, dout


def _check_fwd(inp, W, F, sink, out, lse, dtype, rows=slice(None)):
    cu = inp.cu_seqlens.tolist()
    scale = inp.q.shape[2] ** -0.5
    mask = A.mask_of(cu, W, F, DEV)[rows]
    ref, rlse, bo, bl = A.forward(inp.q[rows], inp.k, inp.v, mask, sink, scale, dtype)
    A.check(out[rows], ref, bo, "out")
    A.check(lse[rows], rlse, bl, "lse")


def _check_bwd(inp, W, F, sink, out, lse, dout, grads, dtype):
    ref = A.backward(inp.q, inp.k, inp.v, out, lse, dout, A.mask_of(inp.cu_seqlens.tolist(), W, F, DEV), sink,
                     inp.q.shape[2] ** -0.5, dtype)
    for g, name in zip(grads, ("dq", "dk", "dv", "dsink")):
        if name in ref:
            assert g.dtype == (F32 if name == "dsink" else dtype)
            A.check(g, *ref[name], name)
        else:
            assert g is None


def _run(docs, H, dk, dv, dtype, W, F, with_sink=True, seed=0, grad=True, path=None):
    inp, dout = _inputs(docs, H, dk, dv, dtype, seed)
    sink = inp.sink if with_sink else None
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, inp.max_seqlen, W, F, sink)
    if path is not None:
        assert hs.last_path() == path[0]
    hs.poll_status()
    _check_fwd(inp, W, F, sink, out, lse, dtype)
    if grad:
        g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, inp.cu_seqlens, inp.max_seqlen, W, F, out, lse, dout, sink)
        if path is not None:
            assert hs.last_path() == path[1]
        hs.poll_status()
        _check_bwd(inp, W, F, sink, out, lse, dout, g, dtype)


WF = [(1, 0), (1, 1), (3, 2), (40, 5), (16, 200), (1000, 7), (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("W,F", WF)
def test_fp32(W, F):
    _run([97, 40, 1, 150], 4, 64, 48, F32, W, F, with_sink=W != 40)


@pytest.mark.parametrize("H,dk,dv", [(1, 1, 1), (3, 40, 24), (5, 33, 70)])
def test_odd_shapes(H, dk, dv):
    for dtype in (F32, BF16):
        _run([33, 2, 60], H, dk, dv, dtype, 9, 3)


@pytest.mark.parametrize("W,F", WF + [(100, 4), (128, 128), (129, 130), (124, 4), (120, 8), (250, 6)])
def test_mla_shape(W, F):
    _run([130, 64, 1, 257], 64, 576, 512, BF16, W, F, with_sink=F != 5, seed=1)


@pytest.mark.parametrize("dk,dv", [(512, 512), (192, 128), (64, 64), (576, 448), (256, 320)])
@pytest.mark.parametrize("W,F", [(30, 4), (200, 17)])
def test_widths(dk, dv, W, F):
    _run([150, 290], 64, dk, dv, BF16, W, F, seed=2)


@pytest.mark.parametrize("docs", [[1], [2], [0, 3, 0], [127], [128], [129, 1], [5] * 60])
def test_document_lengths(docs):
    _run(docs, 64, 128, 128, BF16, 6, 2, seed=3)


def test_several_query_ranges_of_the_backward():
    """A document longer than the backward's query ranges: its first keys get
    gradients from all of them."""
    docs, W, F = [1300, 700], 33, 40
    _run(docs, 64, 64, 64, BF16, W, F, seed=4)


def test_matches_the_oracle():
    docs, W, F = [90, 41], 20, 3
    inp, _ = _inputs(docs, 64, 576, 512, BF16, 5)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, inp.max_seqlen, W, F, inp.sink)
    n = lambda t: t.double().cpu().numpy()
    ref = O.swa_first_mqa_fwd(n(inp.q), n(inp.k), n(inp.v), inp.cu_seqlens.tolist(), W, F, n(inp.sink))
    # out: two roundings of at most 2^-8 over values of size |v| <= 6
    assert np.abs(n(out) - ref["out"]).max() <= 6 * 2 * 2.0 ** -8
    assert np.abs(n(lse) - ref["lse"]).max() <= 1e-4


@pytest.mark.parametrize("shape", [(64, 576, 512), (64, 192, 128), (4, 64, 48)])
def test_nothing_outside_the_key_set_is_used(shape):
    """NaN and infinities between the first tokens and the window, behind the
    query and in other documents; q of the poisoned tokens stays finite."""
    docs, W, F, bad = [200, 150, 60], 20, 5, [30, 31, 77, 128, 260, 350, 351, 409]
    inp, dout = _inputs(docs, *shape, BF16, 6)
    cu = inp.cu_seqlens.tolist()
    for i, t in enumerate(bad):
        inp.k[t], inp.v[t] = (float("nan"), float("inf")) if i % 2 else (float("-inf"), float("nan"))
    mask = A.mask_of(cu, W, F, DEV)
    clean = ~mask[:, bad].any(1)
    assert 200 < int(clean.sum()) < sum(docs)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, inp.max_seqlen, W, F, inp.sink)
    hs.poll_status()
    _check_fwd(inp, W, F, inp.sink, out, lse, BF16, rows=clean)
    # the backward of the rows that stay clean: the other rows are given finite
    # outputs and zero probabilities
    out[~clean], lse[~clean] = 0, float("inf")
    dq = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, inp.cu_seqlens, inp.max_seqlen, W, F, out, lse, dout, inp.sink)[0]
    hs.poll_status()
    ref = A.backward(inp.q[clean], inp.k, inp.v, out[clean], lse[clean], dout[clean], mask[clean], inp.sink,
                     shape[1] ** -0.5, BF16)
    A.check(dq[clean], *ref["dq"], "dq")


def test_strided_and_aliased_inputs():
    docs, W, F = [140, 75], 50, 4
    T = sum(docs)
    base, dout = _inputs(docs, 64, 576, 512, BF16, 7)
    for pad, offset in ((8, 0), (16, 8), (3, 1)):  # the last one is not 16-byte aligned
        q = torch.zeros((T, 66, 576 + pad), device=DEV, dtype=BF16)[:, 1:65, offset:offset + 576]
        kv = torch.zeros((T, 576 + pad), device=DEV, dtype=BF16)[:, offset:offset + 576]
        q.copy_(base.q)
        kv.copy_(base.k)
        v = kv[:, :512]  # the latent part of the keys
        out, lse = hs.hs_swa_first_mqa_fwd(q, kv, v, base.cu_seqlens, 140, W, F, base.sink)
        g = hs.hs_swa_first_mqa_bwd(q, kv, v, base.cu_seqlens, 140, W, F, out, lse, dout, base.sink)
        hs.poll_status()
        base.v = v
        _check_fwd(base, W, F, base.sink, out, lse, BF16)
        _check_bwd(base, W, F, base.sink, out, lse, dout, g, BF16)


def test_wide_window_equals_the_window_call():
    docs = [129, 300]
    inp, _ = _inputs(docs, 64, 192, 128, BF16, 8)
    a = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, 300, 64, 0, inp.sink)
    b = hs.hs_swa_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, 300, 64, inp.sink)
    # both are within the bound of the same values; the roundings are at most two of 2^-8 each
    assert (a[0].float() - b[0].float()).abs().max() <= 4 * 2.0 ** -8 * inp.v.abs().max()
    assert (a[1] - b[1]).abs().max() <= 1e-4


@pytest.mark.parametrize("shape,dtype", [((64, 576, 512), BF16), ((4, 64, 48), F32)])
def test_deterministic_on_another_stream_and_in_a_graph(shape, dtype):
    docs, W, F = [200, 333], 60, 4
    inp, dout = _inputs(docs, *shape, dtype, 9)
    args = (inp.cu_seqlens, inp.max_seqlen, W, F)

    def step():
        out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
        return (out, lse) + tuple(hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink))

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    again = torch.randn_like(inp.q)
    keep = inp.q.clone()
    inp.q.copy_(again)
    graph.replay()
    moved = [x.clone() for x in held]
    fresh = step()
    inp.q.copy_(keep)
    graph.replay()
    hs.poll_status()
    for a, b, c, d, e in zip(want, other, held, moved, fresh):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(d, e)


def test_calls_side_by_side_on_two_streams():
    """Forward and backward of two problems at once, narrow and wide windows, again
    and again: bit for bit what each gives alone."""
    cases = [(_inputs([300, 77, 1], 64, 192, 128, BF16, 22), 300, 20, 3),
             (_inputs([410, 90], 64, 576, 512, BF16, 23), 410, 300, 5)]

    def step(case):
        (inp, dout), longest, W, F = case
        args = (inp.cu_seqlens, longest, W, F)
        out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
        return (out, lse) + tuple(hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink))

    want = [step(c) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(cases[i]))
    torch.cuda.synchronize()
    hs.poll_status()
    for w, runs in zip(want, got):
        for g in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_huge_logits_and_rows_without_weight():
    """Logits of +-3e4 (one key takes everything, others underflow) and a sink
    that takes everything."""
    docs, W, F = [260], 70, 4
    inp, _ = _inputs(docs, 64, 192, 128, BF16, 10)
    inp.q.mul_(1000)
    inp.sink.fill_(2.0)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, 260, W, F, inp.sink)
    hs.poll_status()
    _check_fwd(inp, W, F, inp.sink, out, lse, BF16)
    inp.sink.fill_(1e6)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, 260, W, F, inp.sink)
    assert not out.any() and torch.equal(lse, torch.full_like(lse, 1e6))


def test_malformed_documents_are_reported():
    inp, _ = _inputs([64, 64], 64, 64, 64, BF16, 11)
    out = torch.full((128, 64, 64), 7.0, device=DEV, dtype=BF16)
    cu = torch.tensor([0, 64, 100], device=DEV, dtype=torch.int32)  # the last 28 rows are in no document
    hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, cu, 64, 8, 2, inp.sink, out=out)
    with pytest.raises(hs.HSError) as e:
        hs.poll_status()
    assert e.value.status == hs.HS_ERR_INVALID_ARG
    assert bool((out[100:] == 7).all()) and not bool((out[:100] == 7).all())


def test_backward_reports_malformed_documents():
    """Rows in no document are reported; with a window that computes delta in the
    query pass and with one that does not, the other rows keep their gradients."""
    for W in (8, 400):
        inp, dout = _inputs([400, 128], 64, 64, 512, BF16, 20)
        out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, 400, W, 2, inp.sink)
        hs.poll_status()
        cu = torch.tensor([0, 400, 500], device=DEV, dtype=torch.int32)
        g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, cu, 400, W, 2, out, lse, dout, inp.sink)
        with pytest.raises(hs.HSError) as e:
            hs.poll_status()
        assert e.value.status == hs.HS_ERR_INVALID_ARG
        r = slice(0, 400)
        ref = A.backward(inp.q[r], inp.k[r], inp.v[r], out[r], lse[r], dout[r], A.mask_of([0, 400], W, 2, DEV), None,
                         64 ** -0.5, BF16)
        A.check(g[0][r], *ref["dq"], "dq")


@pytest.mark.parametrize("W", [20, 300])
def test_backward_of_an_output_at_any_element(W):
    """out one element past a 16-byte boundary."""
    docs, F = [330, 41], 4
    inp, dout = _inputs(docs, 64, 64, 512, BF16, 21)
    args = (inp.cu_seqlens, 330, W, F)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
    moved = torch.empty(out.numel() + 8, device=DEV, dtype=BF16)[1:out.numel() + 1].view(out.shape)
    moved.copy_(out)
    g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, moved, lse, dout, inp.sink)
    assert hs.last_path() == hs.HS_PATH_MMA
    hs.poll_status()
    _check_bwd(inp, W, F, inp.sink, out, lse, dout, g, BF16)


def test_no_tokens():
    q = torch.zeros((0, 64, 576), device=DEV, dtype=BF16)
    k, v = q[:, 0], q[:, 0, :512]
    cu, sink = torch.zeros(1, device=DEV, dtype=torch.int32), torch.zeros(64, device=DEV)
    out, lse = hs.hs_swa_first_mqa_fwd(q, k, v, cu, 1, 4, 1, sink)
    assert out.shape == (0, 64, 512) and lse.shape == (0, 64)
    g = hs.hs_swa_first_mqa_bwd(q, k, v, cu, 1, 4, 1, out, lse, out, sink)
    assert g[0].shape == (0, 64, 576) and not g[3].any()


@pytest.mark.parametrize("W,F", [(30, 4), (100, 0), (20, 300)])
def test_a_spoiled_query_spoils_only_its_own_keys(W, F):
    """NaN in a query's q and infinity in another's dout: keys that neither sees
    keep their gradients, in every document.  (20, 300): more first tokens than
    the band takes."""
    docs = [400, 150, 333]
    inp, dout = _inputs(docs, 64, 192, 128, BF16, 12)
    cu = inp.cu_seqlens.tolist()
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, 400, W, F, inp.sink)
    bad = [211, 430]
    inp.q[bad[0], 3, 7] = float("nan")
    dout[bad[1], 60, 100] = float("inf")
    g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, inp.cu_seqlens, 400, W, F, out, lse, dout, inp.sink)
    hs.poll_status()
    mask = A.mask_of(cu, W, F, DEV)
    rows = torch.ones(sum(docs), dtype=torch.bool, device=DEV)
    rows[bad] = False
    keys = ~mask[bad].any(0)
    ref = A.backward(inp.q[rows], inp.k, inp.v, out[rows], lse[rows], dout[rows], mask[rows], None,
                     192 ** -0.5, BF16)
    assert 300 < int(keys.sum()) < sum(docs)
    A.check(g[0][rows], *ref["dq"], "dq")
    for i, name in ((1, "dk"), (2, "dv")):
        A.check(g[i][keys], *(x[keys] for x in ref[name]), name)
    assert bool(g[1][bad[0]].isnan().any()) and not bool(g[2][bad[1]].isfinite().all())


@pytest.mark.parametrize("docs,W,F", [([700, 30, 900], 64, 250), ([1200, 64, 65, 300], 40, 33), ([2100, 90], 300, 5),
                                      ([600], 50, 257), ([128] * 9 + [1], 127, 3), ([513, 511], 512, 1)])
def test_first_tokens_over_chunks_and_documents(docs, W, F):
    """Documents that begin and end inside token chunks and key tiles, first tokens
    up to and past what the band takes."""
    _run(docs, 64, 128, 64, BF16, W, F, seed=13)


def test_other_passes_without_the_band():
    """A workspace that has no room for the band: the window passes' own."""
    docs, W, F = [300, 290], 100, 6
    inp, dout = _inputs(docs, 64, 192, 128, BF16, 14)
    args = (inp.cu_seqlens, 300, W, F)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
    want = hs.workspace_size(hs.HS_OP_SWA_FIRST_MQA_BWD, 590, 2, 300, 64, 192, 128, BF16, W + F)
    with pytest.raises(hs.HSError) as e:
        hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink,
                                workspace=torch.empty(want - 1, dtype=torch.uint8, device=DEV))
    assert e.value.status == hs.HS_ERR_WORKSPACE
    big = torch.full((want + 5000,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN wherever it is read first
    g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink, workspace=big)
    hs.poll_status()
    assert bool((big[want:] == 0xFF).all())
    _check_bwd(inp, W, F, inp.sink, out, lse, dout, g, BF16)


def test_a_workspace_full_of_nan():
    """A window wide enough for delta in the query pass: nothing is read before it is written."""
    docs, W, F = [500, 1, 90], 260, 6
    inp, dout = _inputs(docs, 64, 192, 512, BF16, 24)
    args = (inp.cu_seqlens, 500, W, F)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
    want = hs.workspace_size(hs.HS_OP_SWA_FIRST_MQA_BWD, 591, 3, 500, 64, 192, 512, BF16, W + F)
    ws = torch.full((want + 5000,), 0xFF, dtype=torch.uint8, device=DEV)
    g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink, workspace=ws)
    hs.poll_status()
    assert bool((ws[want:] == 0xFF).all())
    _check_bwd(inp, W, F, inp.sink, out, lse, dout, g, BF16)


def test_a_loose_bound_of_the_lengths():
    """max_seqlen, window and num_first far above the tokens there are."""
    docs, far = [700, 1], 200000
    inp, dout = _inputs(docs, 64, 64, 64, BF16, 16)
    args = (inp.cu_seqlens, far, far, far)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
    g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink)
    hs.poll_status()
    _check_fwd(inp, far, far, inp.sink, out, lse, BF16)
    _check_bwd(inp, far, far, inp.sink, out, lse, dout, g, BF16)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_gradients_at_any_element(which):
    """dq, dk or dv one element past a 16-byte boundary; nothing beside them is written."""
    docs, W, F = [130, 41], 30, 4
    inp, dout = _inputs(docs, 64, 64, 128, BF16, 17)
    args = (inp.cu_seqlens, 130, W, F)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
    grads, holds = [], []
    for i, x in enumerate((inp.q, inp.k, dout[:, 0])):
        off = int(i == which)
        holds.append(torch.full((x.numel() + 16,), 7.0, device=DEV, dtype=BF16))
        grads.append(holds[i][off:off + x.numel()].view(x.shape))
    grads.append(torch.empty(64, device=DEV))
    g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink, grads=grads)
    hs.poll_status()
    _check_bwd(inp, W, F, inp.sink, out, lse, dout, g, BF16)
    for i, h in enumerate(holds):
        off = int(i == which)
        assert bool((h[:off] == 7).all()) and bool((h[off + grads[i].numel():] == 7).all())


def test_many_tokens_in_several_documents():
    """Enough tokens for the backward's longest items, each document checked by itself."""
    docs, W, F = [1300, 3, 1250, 1100, 1290, 260], 70, 9
    inp, dout = _inputs(docs, 64, 64, 128, BF16, 19)
    cu = inp.cu_seqlens.tolist()
    args = (inp.cu_seqlens, 1300, W, F)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
    g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink)
    hs.poll_status()
    for bos, eos in zip(cu, cu[1:]):
        r = slice(bos, eos)
        mask = A.mask_of([0, eos - bos], W, F, DEV)
        ref, rlse, bo, bl = A.forward(inp.q[r], inp.k[r], inp.v[r], mask, inp.sink, 64 ** -0.5, BF16)
        A.check(out[r], ref, bo, "out")
        A.check(lse[r], rlse, bl, "lse")
        ref = A.backward(inp.q[r], inp.k[r], inp.v[r], out[r], lse[r], dout[r], mask, None, 64 ** -0.5, BF16)
        for x, name in zip(g, ("dq", "dk", "dv")):
            A.check(x[r], *ref[name], name)


def test_far_tokens_pass_32_bit_offsets():
    """70000 tokens of the MLA shape, where out, q and the gradients have more than
    2^31 elements: the last rows and keys, and the first tokens' share in them."""
    T, W, F, n = 70000, 100, 4, 300
    g = torch.Generator(device=DEV)
    g.manual_seed(18)
    new = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=BF16)
    q, k, v, dout, sink = new(T, 64, 576), new(T, 576), new(T, 512), new(T, 64, 512), new(64).float()
    args = (torch.tensor([0, T], device=DEV, dtype=torch.int32), T, W, F)
    out, lse = hs.hs_swa_first_mqa_fwd(q, k, v, *args, sink)
    grads = hs.hs_swa_first_mqa_bwd(q, k, v, *args, out, lse, dout, sink)
    hs.poll_status()
    rows = slice(T - n, T)
    keys = torch.cat([torch.arange(F, device=DEV), torch.arange(T - n - W, T, device=DEV)])
    t = torch.arange(T - n, T, device=DEV)[:, None]
    mask = (keys <= t) & ((keys > t - W) | (keys < F))
    ref, rlse, bo, bl = A.forward(q[rows], k[keys], v[keys], mask, sink, 576 ** -0.5, BF16)
    A.check(out[rows], ref, bo, "out")
    A.check(lse[rows], rlse, bl, "lse")
    ref = A.backward(q[rows], k[keys], v[keys], out[rows], lse[rows], dout[rows], mask, None, 576 ** -0.5, BF16)
    A.check(grads[0][rows], *ref["dq"], "dq")
    for i, name in ((1, "dk"), (2, "dv")):  # keys that only these rows attend
        A.check(grads[i][rows], *(x[F + W:] for x in ref[name]), name)


def _check_fwd_by_documents(inp, W, F, out, lse, most):
    """Every row, `most` rows and the keys they may see at a time: documents are
    joined while they fit, longer ones are cut into pieces of rows."""
    cu, scale = inp.cu_seqlens.tolist(), inp.q.shape[2] ** -0.5
    pieces, bos = [], 0  # (first key, first row, end, documents)
    for d in range(1, len(cu)):
        if d + 1 < len(cu) and cu[d + 1] - cu[bos] <= most:
            continue
        pieces += [(cu[bos], r, min(r + most, cu[d]), cu[bos:d + 1]) for r in range(cu[bos], cu[d], most)]
        bos = d
    for key0, r0, r1, ends in pieces:
        rows = slice(r0, r1)
        if len(ends) > 2:
            keys = torch.arange(r0, r1, device=DEV)
            mask = A.mask_of([e - key0 for e in ends], W, F, DEV)
        else:  # the first tokens and what the rows' windows reach
            keys = torch.cat([torch.arange(key0, min(key0 + F, r0), device=DEV),
                              torch.arange(max(min(key0 + F, r0), r0 - W + 1), r1, device=DEV)])
            t = torch.arange(r0, r1, device=DEV)[:, None]
            mask = (keys <= t) & ((keys > t - W) | (keys < key0 + F))
        ref, rlse, bo, bl = A.forward(inp.q[rows], inp.k[keys], inp.v[keys], mask, inp.sink, scale, BF16)
        A.check(out[rows], ref, bo, "out")
        A.check(lse[rows], rlse, bl, "lse")


@pytest.mark.parametrize("docs", [[1, 2, 3, 1, 1] * 1500, [2] * 6000, [1] * 5000])
def test_thousands_of_short_documents(docs):
    """Passes of one tile, many for a pair, where finding the documents takes as long
    as the pass: no role may run away from the others."""
    W, F = 2, 1
    inp, _ = _inputs(docs, 64, 64, 64, BF16, 25)
    for _ in range(5):
        out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, 3, W, F, inp.sink)
        assert hs.last_path() == hs.HS_PATH_TCGEN05
        hs.poll_status()
    _check_fwd_by_documents(inp, W, F, out, lse, 400)


@pytest.mark.parametrize("docs,W,F", [([4096], 300, 4), ([4096], 1000, 8), ([2500, 1, 1500], 256, 0), ([3001], 512, 200)])
def test_many_passes_of_several_tiles(docs, W, F):
    """Two, three and four tiles of 256 keys a pass, many passes for a pair: a row's sum
    is read while the next pass of its CTA may have begun.  Every row, again and again."""
    inp, _ = _inputs(docs, 64, 64, 64, BF16, 26)
    call = lambda: hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, inp.max_seqlen, W, F, inp.sink)
    out, lse = call()
    assert hs.last_path() == hs.HS_PATH_TCGEN05
    hs.poll_status()
    _check_fwd_by_documents(inp, W, F, out, lse, 256)
    for _ in range(20):
        o, l = call()
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("H,dk,dv,dtype,simt", [(4, 64, 48, F32, False), (4, 64, 48, BF16, False),
                                                (64, 192, 128, BF16, False), (64, 192, 128, BF16, True)])
@pytest.mark.parametrize("low", [float("-inf"), -3e38])
def test_first_keys_of_weight_zero(H, dk, dv, dtype, simt, low):
    """A key whose logit is -inf (held, or past fp32) takes no weight, though it is the
    first one alone that a running maximum meets."""
    docs, W, F = [150, 1, 330], 20, 1
    inp, _ = _inputs(docs, H, dk, dv, dtype, 27)
    cu = inp.cu_seqlens.tolist()
    inp.q[:, :, 0] = 1000.0
    inp.k[:, 0] = 0.0
    inp.k[cu[:-1], 0] = low
    hs.set_force_simt(simt)
    try:
        out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, 330, W, F, inp.sink)
    finally:
        hs.set_force_simt(False)
    hs.poll_status()
    mask = A.mask_of(cu, W, F, DEV)
    mask[:, cu[:-1]] = False
    ref, rlse, bo, bl = A.forward(inp.q, inp.k, inp.v, mask, inp.sink, dk ** -0.5, dtype)
    A.check(out, ref, bo, "out")
    A.check(lse, rlse, bl, "lse")


def test_a_first_segment_of_weight_zero():
    """The same for the first 128 keys of a window and for a first selected block."""
    T, H, dk, dv, W = 300, 4, 64, 48, 260
    inp, _ = _inputs([T], H, dk, dv, F32, 28)
    inp.q[:, :, 0] = 1000.0
    inp.k[:, 0] = 0.0
    inp.k[:200, 0] = float("-inf")
    rows, t = slice(250, T), torch.arange(250, T, device=DEV)[:, None]
    j = torch.arange(T, device=DEV)
    out, lse = hs.hs_swa_mqa_fwd(inp.q, inp.k, inp.v, inp.cu_seqlens, T, W, inp.sink)
    hs.poll_status()
    ref, rlse, bo, bl = A.forward(inp.q[rows], inp.k, inp.v, (j <= t) & (j >= 200), inp.sink, dk ** -0.5, F32)
    A.check(out[rows], ref, bo, "out")
    A.check(lse[rows], rlse, bl, "lse")
    idx = torch.stack([torch.zeros_like(j), j // 16], 1).int()
    idx[:16, 1] = -1
    out, lse = hs.hs_sparse_mqa_fwd(inp.q, inp.k, inp.v, idx, inp.cu_seqlens, T, 16, inp.sink)
    hs.poll_status()
    ref, rlse, bo, bl = A.forward(inp.q[rows], inp.k, inp.v, (j <= t) & (j // 16 == t // 16), inp.sink, dk ** -0.5, F32)
    A.check(out[rows], ref, bo, "out")
    A.check(lse[rows], rlse, bl, "lse")


def _graph_nodes(call):
    """Kernels that call() launches."""
    call()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = ctypes.c_size_t()
    assert ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


def test_a_window_past_the_documents_takes_the_same_kernels():
    """Where delta is computed goes by the keys that a token can attend, not by the
    window's number: packed short documents with a window that holds each of them."""
    docs, F = [60, 33, 64, 7] * 6, 4
    inp, dout = _inputs(docs, 64, 64, 512, BF16, 29)
    nodes, grads = [], []
    for W in (64, 512, 2 ** 31 - 1):
        args = (inp.cu_seqlens, 64, W, F)
        out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
        call = lambda: hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink)
        nodes.append(_graph_nodes(call))
        grads.append(call())
    hs.poll_status()
    assert nodes[0] == nodes[1] == nodes[2]
    for g in grads[1:]:
        assert all(torch.equal(a, b) for a, b in zip(g, grads[0]))


def test_a_band_past_its_limit():
    """P and dS of every key would take more than the workspace may: the passes that
    compute them again, for the last rows and the keys that only those attend."""
    T, W, F, n = 8192, 2100, 4, 300
    size = lambda W: hs.workspace_size(hs.HS_OP_SWA_FIRST_MQA_BWD, T, 1, T, 64, 64, 64, BF16, W + F)
    assert size(W) < 2 ** 30 < 2 ** 31 < size(1500)
    inp, dout = _inputs([T], 64, 64, 64, BF16, 30)
    args = (inp.cu_seqlens, T, W, F)
    out, lse = hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink)
    g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink)
    assert hs.last_path() == hs.HS_PATH_MMA
    hs.poll_status()
    rows = slice(T - n, T)
    keys = torch.cat([torch.arange(F, device=DEV), torch.arange(T - n - W, T, device=DEV)])
    t = torch.arange(T - n, T, device=DEV)[:, None]
    mask = (keys <= t) & ((keys > t - W) | (keys < F))
    ref = A.backward(inp.q[rows], inp.k[keys], inp.v[keys], out[rows], lse[rows], dout[rows], mask, None, 64 ** -0.5,
                     BF16)
    A.check(g[0][rows], *ref["dq"], "dq")
    for i, name in ((1, "dk"), (2, "dv")):
        A.check(g[i][rows], *(x[F + W:] for x in ref[name]), name)
    # the sink's gradient from every row
    terms = torch.exp(inp.sink.double() - lse.double()) * (dout.double() * out.double()).sum(-1)
    u = 2.0 ** -20 * (1 + lse.abs() + inp.sink.abs()) + (T + 64) * 2.0 ** -23
    size = (torch.exp(inp.sink.double() - lse.double()) * (dout.double() * out.double()).abs().sum(-1))
    A.check(g[3], -terms.sum(0), (u * size).sum(0), "dsink")


def test_no_tokens_through_the_c_call():
    """dsink is the one output with elements."""
    dsink, p = torch.full((64,), 7.0, device=DEV), torch.zeros(64, device=DEV)
    at = ctypes.c_void_p(p.data_ptr())
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    st = hs.lib().hs_swa_first_mqa_bwd(at, 64 * 576, 576, at, 576, at, 512, at, 0, 0, 0, 64, 576, 512, hs.HS_BF16, 0.0,
                                       16, 2, at, at, at, at, at, at, at, ctypes.c_void_p(dsink.data_ptr()), None, 0,
                                       stream)
    assert st == hs.HS_OK and not dsink.any()


@pytest.mark.parametrize("W", [8, 400])
@pytest.mark.parametrize("cu,most,good", [([0, 400, 500], 400, [(0, 400), (400, 500)]),  # the last 28 rows in none
                                          ([5, 400, 528], 400, [(5, 400), (400, 528)]),  # the first 5 in none
                                          ([0, 151, 451, 528], 200, [(0, 151), (451, 528)])])  # one past the bound
def test_rows_in_no_document_give_nothing_to_the_others(W, cu, most, good):
    """Their part of the workspace is never taken for probabilities: dq, dk, dv of the
    documents that are right, and dsink from those rows alone."""
    F, T, stale = 2, 528, 0x3C  # bf16 0x3C3C is 0.0115
    inp, dout = _inputs([T], 64, 64, 512, BF16, 31)
    args = (torch.tensor(cu, device=DEV, dtype=torch.int32), most, W, F)
    out, lse = torch.zeros((T, 64, 512), device=DEV, dtype=BF16), torch.full((T, 64), 1.0, device=DEV)
    hs.hs_swa_first_mqa_fwd(inp.q, inp.k, inp.v, *args, inp.sink, out=out, lse=lse)
    with pytest.raises(hs.HSError):
        hs.poll_status()
    need = hs.workspace_size(hs.HS_OP_SWA_FIRST_MQA_BWD, T, len(cu) - 1, most, 64, 64, 512, BF16, min(W, most) + F)
    ws = torch.full((need,), stale, dtype=torch.uint8, device=DEV)
    g = hs.hs_swa_first_mqa_bwd(inp.q, inp.k, inp.v, *args, out, lse, dout, inp.sink, workspace=ws)
    assert hs.last_path() == hs.HS_PATH_MMA
    with pytest.raises(hs.HSError) as e:
        hs.poll_status()
    assert e.value.status == hs.HS_ERR_INVALID_ARG
    dsink, room = torch.zeros(64, device=DEV, dtype=torch.float64), 0.0
    for a, b in good:
        r = slice(a, b)
        ref = A.backward(inp.q[r], inp.k[r], inp.v[r], out[r], lse[r], dout[r], A.mask_of([0, b - a], W, F, DEV),
                         inp.sink, 64 ** -0.5, BF16)
        for x, name in zip(g, ("dq", "dk", "dv")):
            A.check(x[r], *ref[name], name)
        dsink, room = dsink + ref["dsink"][0], room + ref["dsink"][1]
    A.check(g[3], dsink, room, "dsink")


def test_without_tensor_cores():
    """The CUDA-core kernels at the shape that normally does not reach them."""
    hs.set_force_simt(True)
    try:
        _run([90, 41, 1], 64, 192, 128, BF16, 20, 3, seed=15, path=(hs.HS_PATH_SIMT, hs.HS_PATH_SIMT))
    finally:
        hs.set_force_simt(False)
    _run([90, 41, 1], 64, 192, 128, BF16, 20, 3, seed=15, path=(hs.HS_PATH_TCGEN05, hs.HS_PATH_MMA))
