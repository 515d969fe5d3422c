"""Plain 64-bit forms of the windowed operators for the GPU tests, and the bounds their outputs are held to.

Every bound is per element and follows from where the kernels round (u = 2^-8 is half a bf16 step relative to the
value, e = 2^-24 half an fp32 step):

* a score is an fp32 sum of d exact products: |S - S64| <= (d + 2) e |Q||K|^T scale =: eS;
* P_bar is rounded to bf16 before P V, the row sum is not: |O - O64| <= (u + eP) (P|V| + |O|) + u |O|, with eP the
  relative error that eS, ex2.approx (2^-22) and the fp32 sums give a probability;
* the backward rounds P to bf16 before P^T dO, dS to bf16 before dS K and dS^T Q, and the results to bf16; dP and
  delta are fp32 sums of d products.

Second-order terms are covered by the factor SLACK.
"""

import math

import torch

U, E, SLACK = 2.0 ** -8, 2.0 ** -24, 1.02


def visible(N, window, sinks, device):
    at = torch.arange(N, device=device)
    i, j = at[:, None], at[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def attention(q, k, v, seen):
    """64-bit attention of q [.., T, d] over k, v [.., L, d] where `seen` [.., T, L]; rows that see nothing give 0
    and -inf.  Returns o, lse, P and the bounds of o and lse."""
    q, k, v = q.double(), k.double(), v.double()
    d, L = q.shape[-1], k.shape[-2]
    scale = 1.0 / math.sqrt(d)
    x = (q @ k.transpose(-1, -2) * scale).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    o = p @ v
    es = ((d + 2) * E * scale * (q.abs() @ k.abs().transpose(-1, -2)) + 4 * E * x.abs()).masked_fill(~seen, 0.0)
    top = es.amax(-1, keepdim=True) if L else es.new_zeros(*es.shape[:-1], 1)
    # probability: its own score, the shift, the sum of the others, ex2, the fp32 sum of up to L terms (kept in
    # at least 64 partial sums per row) and of the products
    ep = 2 * (es + top) + 2.0 ** -21 + (L / 32 + 16) * E
    o_bound = SLACK * (((p * (U + ep)) @ v.abs()) + (U + ep.amax(-1, keepdim=True)) * o.abs()) if L else o.abs()
    # a probability below the smallest normal number of bf16 relative to its row's shift is lost whole
    o_bound = o_bound + 2.0 ** -60 * v.abs().amax(-2, keepdim=True) if L else o_bound
    lse_bound = SLACK * (2 * top[..., 0] + 2.0 ** -20 + (L / 32 + 16) * E + 4 * E * torch.where(torch.isinf(lse), 0.0, lse).abs())
    return {"o": o, "lse": lse, "p": p, "es": es, "ep": ep, "o_bound": o_bound, "lse_bound": lse_bound}


def gradients(q, k, v, o, do, f, lse_bound):
    """64-bit gradients for delta taken from the given o, with `f` from attention(); returns values and bounds."""
    q, k, v, o, do = (t.double() for t in (q, k, v, o, do))
    d, L, T = q.shape[-1], k.shape[-2], q.shape[-2]
    scale = 1.0 / math.sqrt(d)
    p = f["p"]
    ep = p * (2 * f["es"] + lse_bound[..., None] + 2.0 ** -20)  # error of the recomputed fp32 probability
    delta = (do * o).sum(-1, keepdim=True)
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - delta)
    edp = (d + 2) * E * (do.abs() @ v.abs().transpose(-1, -2)) + (d + 2) * E * (do.abs() * o.abs()).sum(-1, keepdim=True)
    e32 = ep * (dp - delta).abs() + p * (edp + 4 * E * (dp.abs() + delta.abs()))
    eds = e32 + U * (ds.abs() + e32)
    acc = (max(L, T) / 16 + 16) * E  # fp32 accumulation of products, in pieces of 16 at least
    dq, dk, dv = ds @ k * scale, ds.transpose(-1, -2) @ q * scale, p.transpose(-1, -2) @ do
    bq = (eds + acc * ds.abs()) @ k.abs() * scale
    bk = (eds + acc * ds.abs()).transpose(-1, -2) @ q.abs() * scale
    bv = (ep + (U + acc) * (p + ep)).transpose(-1, -2) @ do.abs()
    return {"dq": dq, "dk": dk, "dv": dv, "dq_bound": bq, "dk_bound": bk, "dv_bound": bv}


def rounded(bound, value):
    """The bound of a result that is rounded to bf16 at the end."""
    return SLACK * (bound + U * (value.abs() + bound)) + 2.0 ** -120


def assert_within(name, got, ref, bound):
    got = got.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    same = got == ref  # infinities of empty rows
    err = torch.where(same, 0.0, (got - ref).abs())
    bad = ~(err <= bound)
    if bad.any():
        at = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} elements out of bound, first at {at}: "
                             f"got {float(got[at])!r}, expected {float(ref[at])!r} +- {float(bound.expand_as(err)[at])!r}")
