"""Attention over a boolean mask in float64 with, beside every value, a bound on
how far a kernel that keeps fp32 sums may be from it.

Roundings counted, u = eps / 2 of the tensors' type (2^-8 bf16, 2^-24 fp32; a
fp32 kernel keeps the probabilities in fp32):
  logits      an fp32 sum of dk products may lose 2^-23 of scale * sum |q k| per
              term; exp2 / log2 approximations and the argument's own rounding,
              2^-20 (1 + |s|)
  out         p is rounded once (u), the sum over n keys is fp32, the result is
              rounded once (u)
  gradients   p and ds are rounded once (u) before the products they enter, the
              sums are fp32, the result is rounded once (u)
"""

import torch


def _u(dtype):
    return torch.finfo(dtype).eps / 2


def mask_of(cu, window, first, device="cpu"):
    """[T, T] of the window with visible first tokens."""
    T = int(cu[-1])
    j = torch.arange(T, device=device)
    m = torch.zeros((T, T), dtype=torch.bool, device=device)
    for bos, eos in zip(cu, cu[1:]):
        t = torch.arange(bos, eos, device=device)[:, None]
        m[bos:eos] = (j >= bos) & (j <= t) & ((j > t - window) | (j < bos + first))
    return m


def _logits(q, k, mask, scale):
    """s [T, H, N] and the bound on its error, -inf outside the mask."""
    s = torch.einsum("thd,jd->thj", q, k) * scale
    big = torch.einsum("thd,jd->thj", q.abs(), k.abs()) * scale
    e = q.shape[-1] * 2.0 ** -23 * big + 2.0 ** -20 * (1 + s.abs())
    return s.masked_fill(~mask, -torch.inf), e.masked_fill(~mask, 0.0)


def _in_mask(x, mask):
    """x [N, d] with zeros in rows no query sees (they may hold NaN)."""
    return torch.where(mask.reshape(-1, mask.shape[-1]).any(0)[:, None], x.double(), 0.0)


def forward(q, k, v, mask, sink, scale, dtype):
    """q [T, H, Dk], k [N, Dk], v [N, Dv], mask [T, N] -> out, lse and their bounds."""
    q, k, v, mask = q.double(), _in_mask(k, mask), _in_mask(v, mask), mask[:, None]
    s, es = _logits(q, k, mask, scale)
    e = es.amax(-1)
    lse = torch.logsumexp(s, -1)
    if sink is not None:
        lse = torch.logaddexp(lse, sink.double().expand_as(lse))
    p = torch.where(lse[..., None] > -torch.inf, torch.exp(s - lse[..., None]), 0.0)
    out = torch.einsum("thj,jd->thd", p, v)
    size = torch.einsum("thj,jd->thd", p, v.abs())
    u = _u(dtype)
    n = mask.sum(-1).amax().item()
    # an error e of every logit moves p by 2 e (its own and the sum's)
    bound = size * (u * (dtype != torch.float32) + 2 * e[..., None] + n * 2.0 ** -23) + u * out.abs()
    return out, lse, bound + 1e-30, e + n * 2.0 ** -24 + 2.0 ** -20 * (1 + lse.abs().nan_to_num(0, 0, 0))


def backward(q, k, v, out, lse, dout, mask, sink, scale, dtype):
    """Gradients as functions of the given out and lse: {name: (value, bound)}."""
    q, k, v, do = q.double(), _in_mask(k, mask), _in_mask(v, mask), dout.double()
    o, l, mask = out.double(), lse.double(), mask[:, None]
    s, es = _logits(q, k, mask, scale)
    p = torch.exp(s - l[..., None])
    es = es + 2.0 ** -20 * (1 + l.abs()[..., None])
    delta = (do * o).sum(-1, keepdim=True)
    dv_ = v.shape[-1]
    ed = dv_ * 2.0 ** -23 * (torch.einsum("thd,jd->thj", do.abs(), v.abs())
                             + (do.abs() * o.abs()).sum(-1, keepdim=True))
    ds = p * (torch.einsum("thd,jd->thj", do, v) - delta)
    u, f = _u(dtype), float(dtype != torch.float32)
    n = 2.0 ** -23 * p.shape[0] * p.shape[1]  # terms of the longest sum
    eds = ds.abs() * (u * f + es + n) + p * ed
    ep = p * (u * f + es + n)
    got = {"dq": (torch.einsum("thj,jd->thd", ds, k) * scale, torch.einsum("thj,jd->thd", eds, k.abs()) * scale),
           "dk": (torch.einsum("thj,thd->jd", ds, q) * scale, torch.einsum("thj,thd->jd", eds, q.abs()) * scale),
           "dv": (torch.einsum("thj,thd->jd", p, do), torch.einsum("thj,thd->jd", ep, do.abs()))}
    got = {k_: (g, b + u * g.abs() + 1e-30) for k_, (g, b) in got.items()}
    if sink is not None:
        ps = torch.exp(sink.double() - l)
        d = delta[..., 0]
        ee = (2.0 ** -20 * (1 + l.abs() + sink.double().abs()) + p.shape[0] * 2.0 ** -23) * ps * d.abs() \
            + ps * dv_ * 2.0 ** -23 * (do.abs() * o.abs()).sum(-1)
        got["dsink"] = (-(ps * d).sum(0), ee.sum(0) + 1e-30)
    return got


def check(got, ref, bound, what):
    g = got.double()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    same = (g == ref) | ((g - ref).abs() <= bound)
    if not bool(same.all()):
        i = int((~same).flatten().nonzero()[0])
        raise AssertionError("%s: %d of %d outside the bound, first at %d: %r, expected %r +- %r" % (
            what, int((~same).sum()), same.numel(), i, float(g.flatten()[i]), float(ref.flatten()[i]),
            float(bound.expand_as(ref).flatten()[i])))
