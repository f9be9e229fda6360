"""Gradients of windowed attention, block by block, against the error that independent roundings add up to.

An element's worst case grows with the number of rows that it sums, its value and its error with the root of it: a sink's dK
over thousands of rows could be missing a tile of them and stay within the worst case.  Here the norm of a block's error is
held against the root of the summed squares of what each rounding can do (U = 2^-8, half a step of bf16):

* dS is a bf16 operand, its factor P in fp32: U |dS|, and 2^-10 |dS| for P (its score, its row's LSE) and fp32;
* delta = dO . O with the stored O: O's rounding U |dO O| a column, its P's U |P dP| a key, and fp32 with what the first
  128 positions' sum P dP has instead: 2^-10 sum P |dP|.  Off by e for the row, it moves dS by P e for all of its keys;
* P is a bf16 operand of dV: U P, and 2^-11 P;
* what is common to a row or to all of them (LSE): 2^-11 of the gradient itself; a gradient stored in bf16: U of it.

A rounding is spread evenly over its half step or less, so that a block's error lies near 0.4 of that root; twice the root
is allowed.  A single term cannot exceed it, nor can four that conspire.
"""
import math

import pytest
import torch

from helpers import cuda_or_skip
from test_window import WINDOWS
from window_ref import U, attend, visible

SCALE = 0.11


def _heads(t, Hkv):
    """Adds the query heads of each key head: [B, Hq, n, D] -> [B, Hkv, n, D]."""
    B, Hq, n, D = t.shape
    return t.view(B, Hkv, Hq // Hkv, n, D).sum(2)


def spread_reference(q, k, v, dO, window, sinks, scale):
    """The gradients in 64 bits and, for each, the summed squares of its roundings' sizes."""
    Hkv, Nk, Nq = k.shape[1], k.shape[2], q.shape[2]
    G = q.shape[1] // Hkv
    q, k, v, dO = (t.double() for t in (q, k, v, dO))
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    seen = visible(torch.arange(Nk - Nq, Nk, device=q.device), Nk, window, sinks)
    O, _, P, _ = attend(q, kk, vv, seen, scale)
    PdP = P * torch.matmul(dO, vv.transpose(-1, -2))
    delta = PdP.sum(-1, keepdim=True)
    e2 = (U * PdP).square().sum(-1, keepdim=True) + (U * dO * O).square().sum(-1, keepdim=True) \
        + (2.0 ** -10 * PdP.abs().sum(-1, keepdim=True)).square()
    dS = PdP - P * delta
    dS2, P2, T = ((U + 2.0 ** -10) * dS).square(), P.square(), (-1, -2)
    out = {"P": P, "dS": dS, "PdP": PdP, "q": q, "k": kk, "dO": dO}
    out["dq"] = torch.matmul(dS, kk) * scale
    out["dk"] = _heads(torch.matmul(dS.transpose(*T), q), Hkv) * scale
    out["dv"] = _heads(torch.matmul(P.transpose(*T), dO), Hkv)
    var = {"dq": (torch.matmul(dS2, kk.square()) + e2 * torch.matmul(P, kk).square()) * scale ** 2,
           "dk": _heads(torch.matmul((dS2 + P2 * e2).transpose(*T), q.square()), Hkv) * scale ** 2,
           "dv": _heads(torch.matmul(((U + 2.0 ** -11) * P).square().transpose(*T), dO.square()), Hkv)}
    for n in ("dq", "dk", "dv"):
        out[n + "_var"] = var[n] + (2.0 ** -11 * out[n]).square()
    return out


def blocks(name, n, sinks):
    """128-row tiles of dQ; of dK and dV the sinks, and 128-key tiles without them."""
    if name == "dq":
        return [(r, min(n, r + 128)) for r in range(0, n, 128)]
    out = [(0, min(n, sinks))] if sinks else []
    return out + [(max(t, sinks), min(n, t + 128)) for t in range(0, n, 128) if max(t, sinks) < min(n, t + 128)]


def worst_block(name, got, ref, sinks):
    """The largest ratio of a block's error to what it may be."""
    var = ref[name + "_var"] + ((U * ref[name]).square() if got.dtype == torch.bfloat16 else 0.0)
    err = (got.double() - ref[name]).square()
    assert torch.isfinite(err).all(), name
    worst = 0.0
    for a, b in blocks(name, got.shape[2], sinks):
        e, w = (t[:, :, a:b].sum((2, 3)).sqrt() for t in (err, var))
        assert not (e[w == 0] > 0).any(), f"{name}: rows {a}..{b} are not 0"
        if (w > 0).any():
            worst = max(worst, float((e / (2 * w))[w > 0].max()))
    return worst


# ------------------------------------------------------------------ no GPU: what the check accepts and rejects
def _bf16(t):
    return t.to(torch.bfloat16).double()


def _cpu_case(case):
    B, Hq, Hkv, Nq, Nk, D, window, sinks = case
    g = torch.Generator().manual_seed(sum(case))
    q, k, v, dO = (torch.randn(s, generator=g).bfloat16() for s in ((B, Hq, Nq, D), (B, Hkv, Nk, D), (B, Hkv, Nk, D),
                                                                     (B, Hq, Nq, D)))
    return q, k, v, dO, spread_reference(q, k, v, dO, window, sinks, SCALE)


CPU = [(1, 8, 2, 1999, 1999, 64, 64, 4), (1, 4, 2, 1500, 1500, 64, 64, 4), (1, 4, 4, 2000, 2100, 40, 60, 16),
       (1, 4, 2, 2000, 2000, 80, 100, 300), (1, 2, 1, 300, 300, 64, 40, 0)]


@pytest.mark.parametrize("case", CPU)
def test_block_check_accepts_roundings_and_rejects_mistakes(case):
    q, k, v, dO, ref = _cpu_case(case)
    Hkv, Nq, Nk, window, sinks = k.shape[1], case[3], case[4], case[6], case[7]
    off = Nk - Nq
    # the library's arithmetic: dS rounded once, delta from a rounded O but for the first positions
    seen_v = v.double().repeat_interleave(q.shape[1] // Hkv, 1)
    stored = (ref["dO"] * _bf16(torch.matmul(_bf16(ref["P"]), seen_v))).sum(-1, keepdim=True)
    early = (torch.arange(off, Nk) < 128)[:, None]
    delta = torch.where(early, ref["PdP"].sum(-1, keepdim=True), stored)
    dS = _bf16(ref["PdP"] - ref["P"] * delta)

    def dk_of(x):
        return _heads(torch.matmul(x.transpose(-1, -2), ref["q"]), Hkv) * SCALE

    def dv_of(x):
        return _heads(torch.matmul(x.transpose(-1, -2), ref["dO"]), Hkv)

    good = {"dq": torch.matmul(dS, ref["k"]) * SCALE, "dk": dk_of(dS), "dv": dv_of(_bf16(ref["P"]))}
    for n, t in good.items():
        assert 0.01 < worst_block(n, t, ref, sinks) < 0.5, n
        assert 0.01 < worst_block(n, t.to(torch.bfloat16), ref, sinks) < 0.5, n
    if sinks:
        far = (torch.arange(off, Nk) >= 128 * ((sinks + 127) // 128) + window)[:, None]  # rows behind the sink tiles' windows
        tile = ((torch.arange(Nq) // 128) == (Nq // 2) // 128)[:, None]
        for wrong in (torch.where(far, _bf16(ref["PdP"]), dS), torch.where(far, 1.1 * dS, dS), torch.where(tile, 0.0, dS)):
            only = ref["dk"].clone()  # the mistake in the sinks' dK alone
            only[:, :, :sinks] = dk_of(wrong)[:, :, :sinks]
            assert worst_block("dk", only, ref, sinks) > 1
        only = ref["dv"].clone()
        only[:, :, :sinks] = dv_of(torch.where(tile, 0.0, ref["P"]))[:, :, :sinks]
        assert worst_block("dv", only, ref, sinks) > 1
    assert worst_block("dq", torch.matmul(torch.where(early, dS, _bf16(ref["PdP"])), ref["k"]) * SCALE, ref, sinks) > 1
    assert worst_block("dk", dk_of(torch.where(early, dS, _bf16(ref["PdP"]))), ref, sinks) > 1


# ------------------------------------------------------------------ GPU
CASES = WINDOWS + [(1, 4, 2, 1500, 1500, 128, 64, 4), (1, 4, 2, 1500, 1500, 64, 64, 4), (2, 3, 1, 1700, 1800, 256, 60, 200),
                   (1, 6, 2, 2000, 2000, 80, 100, 300), (1, 2, 2, 2000, 4000, 40, 30, 7), (1, 128, 32, 1999, 1999, 64, 64, 4),
                   (2, 64, 64, 2000, 2100, 40, 60, 16), (1, 4, 2, 700, 900, 192, 100, 200), (1, 6, 2, 1500, 1500, 192, 64, 140),
                   (1, 2, 1, 600, 600, 168, 130, 300), (1, 8, 2, 1999, 1999, 128, 64, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_window_backward_spread(case, grad_dtype):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, Nq, Nk, D, window, sinks = case
    g = torch.Generator(device="cuda")
    g.manual_seed(2 + sum(case))
    q, k, v, dO = (torch.randn(B, h, n, D, generator=g, device="cuda").bfloat16()
                   for h, n in ((Hq, Nq), (Hkv, Nk), (Hkv, Nk), (Hq, Nq)))
    ref = spread_reference(q, k, v, dO, window, sinks, SCALE)
    o, lse = fa.fa_window_forward(q, k, v, window, sinks, scale=SCALE)
    dq, dk, dv, _ = fa.fa_window_backward(q, k, v, o, dO, lse, window, sinks, scale=SCALE, grad_dtype=grad_dtype)
    assert fa.fa_device_status() == 0
    ratios = {n: worst_block(n, t, ref, sinks) for n, t in (("dq", dq), ("dk", dk), ("dv", dv))}
    print(case, {n: f"{r:.3f}" for n, r in ratios.items()})
    assert max(ratios.values()) <= 1, ratios
