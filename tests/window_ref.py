"""Windowed and shared-prefix attention in 64 bits, written from the definition, with a bound on what the
library's roundings can do to every element.

A rounding to bf16 is off by at most half a step, U = 2^-8 of the value.  With A = sum_j P_ij |v_j|:

* O: P is a bf16 operand (U A), O is stored in bf16 (U |O|).  The rest is fp32: a score of D products is off by
  less than D 2^-24 sum|q k| scale (below 2^-13 for these inputs), 2^x by 2^-22 of its value, a sum of n keys'
  products (16 at a time) by n/16 2^-24 A (below 2^-13 up to n = 32768); together below 2^-11 A.
* LSE: the score's error, the sum's, and fp32 at magnitude below 32 (2^-20): below 2^-12.
* delta uses the stored O (but for the first 128 positions): off by at most E = sum_d |dO| bound(O), plus fp32 (2^-16 sum|dO O|).
* dV: P as a bf16 operand, with the LSE's error in it: (U + 2^-11) sum_i P |dO|.
* dS = P (dP - delta) is a bf16 operand, and one kernel takes the bf16 P as its factor:
  (2 U + 2^-10) |dS| + P E; dQ adds it against |k|, dK against |q|.
* gradients stored in bf16 add U of their value.
"""
import math

import torch

U = 2.0 ** -8


def visible(pos, n, window, sinks):
    """[rows, n] mask: position p sees key j iff j <= p and (j < sinks or j > p - window)."""
    p, j = pos[:, None], torch.arange(n, device=pos.device)[None]
    return (j <= p) & ((j < sinks) | (j > p - window))


def attend(q, k, v, seen, scale):
    """O, LSE, P, sum P|v| of q [.., n, D] over k, v [.., m, D]; a row that sees nothing gives O = 0, LSE = -inf."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = e.sum(-1, keepdim=True)
    P = e / torch.where(l == 0, torch.ones_like(l), l)
    lse = torch.where(l == 0, torch.full_like(l, -math.inf), m + torch.log(torch.where(l == 0, torch.ones_like(l), l)))
    return torch.matmul(P, v), lse[..., 0], P, torch.matmul(P, v.abs())


def bound_o(O, A):
    return (U + 2.0 ** -11) * A + U * O.abs()


LSE_TOL = 2.0 ** -12


def window_reference(q, k, v, window, sinks, scale, dO=None):
    """Reference and bounds for q [B, Hq, Nq, D] as the last positions of k, v [B, Hkv, Nk, D]."""
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1:3]
    G = Hq // Hkv
    q, k, v = (t.double() for t in (q, k, v))
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    pos = torch.arange(Nk - Nq, Nk, device=q.device)
    O, lse, P, A = attend(q, kk, vv, visible(pos, Nk, window, sinks), scale)
    out = {"o": O, "lse": lse, "o_bound": bound_o(O, A)}
    if dO is None:
        return out
    dO = dO.double()
    delta = (dO * O).sum(-1, keepdim=True)
    E = (dO.abs() * out["o_bound"]).sum(-1, keepdim=True) + 2.0 ** -16 * (dO * O).abs().sum(-1, keepdim=True)
    dS = P * (torch.matmul(dO, vv.transpose(-1, -2)) - delta)
    err = (2 * U + 2.0 ** -10) * dS.abs() + P * E

    def heads(t):  # add the query heads of each key head
        return t.view(B, Hkv, G, Nk, D).sum(2)

    T = (-1, -2)
    out["delta"], out["delta_bound"] = delta[..., 0], E[..., 0]
    out["dq"], out["dq_bound"] = torch.matmul(dS, kk) * scale, torch.matmul(err, kk.abs()) * scale
    out["dk"], out["dk_bound"] = (heads(torch.matmul(x.transpose(*T), y)) * scale for x, y in ((dS, q), (err, q.abs())))
    out["dv"], out["dv_bound"] = (heads(torch.matmul(P.transpose(*T), y)) * c for y, c in ((dO, 1.0), (dO.abs(), U + 2.0 ** -11)))
    return out


def cached_reference(q, k, v, lens, window, sinks, scale, kp=None, vp=None):
    """Reference for the newest rows q [B, Hq, n_q, D] of sequences that hold lens[b] keys of k, v [B, Hkv, N, D]
    behind an optional prefix kp, vp [Hkv, P, D] that every row sees."""
    B, Hq, n_q, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out = {"o": [], "lse": [], "o_bound": []}
    for b in range(B):
        n = int(lens[b])
        pos = torch.arange(n - n_q, n, device=q.device)
        seen = visible(pos, n, window, sinks)
        kb, vb = k[b, :, :n].double(), v[b, :, :n].double()
        if kp is not None:
            kb, vb = torch.cat((kp.double(), kb), 1), torch.cat((vp.double(), vb), 1)
            seen = torch.cat((torch.ones(n_q, kp.shape[1], dtype=torch.bool, device=q.device), seen), 1)
        if kb.shape[1] == 0:
            kb, vb = (torch.zeros(Hkv, 1, D, dtype=torch.float64, device=q.device) for _ in range(2))
            seen = torch.zeros(n_q, 1, dtype=torch.bool, device=q.device)
        O, L, _, A = attend(q[b].double(), kb.repeat_interleave(G, 0), vb.repeat_interleave(G, 0), seen, scale)
        for name, t in (("o", O), ("lse", L), ("o_bound", bound_o(O, A))):
            out[name].append(t)
    return {n: torch.stack(t) for n, t in out.items()}


def check(got, ref, bound, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    over = (got - ref).abs() - bound
    worst = float(over.max())
    assert worst <= 0, (f"{what}: over its bound by {worst:.3e} at "
                        f"{[int(x) for x in torch.unravel_index(over.argmax(), over.shape)]}; "
                        f"max |err| {float((got - ref).abs().max()):.3e}, {int((over > 0).sum())} elements")


def check_lse(got, ref, what):
    empty = ref == -math.inf
    assert torch.equal(got == -math.inf, empty), f"{what}: rows that see nothing"
    d = (got.double() - ref)[~empty].abs()
    assert d.numel() == 0 or (torch.isfinite(d).all() and float(d.max()) <= LSE_TOL), f"{what}: {float(d.max()):.3e}"
