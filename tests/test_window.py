"""Windowed attention (forward, backward, single tokens) and shared-prefix decode against the definition in 64 bits,
through the library's Python entry points; refusals through the C ABI."""
import ctypes
import math

import pytest
import torch

from attention_tiled_fwd_gb300 import _native as nat
from helpers import cuda_or_skip
from window_ref import (U, attend, cached_reference, check, check_lse, visible, window_reference)


# ------------------------------------------------------------------ no GPU: the reference, and refusals
def test_visible_rows_by_hand():
    # 3 rows at positions 4..6 of 7 keys, window 2, 1 sink
    m = visible(torch.arange(4, 7), 7, 2, 1).int().tolist()
    assert m == [[1, 0, 0, 1, 1, 0, 0], [1, 0, 0, 0, 1, 1, 0], [1, 0, 0, 0, 0, 1, 1]]


def test_reference_rows_that_see_nothing():
    z = torch.zeros(2, 3, dtype=torch.float64)
    O, lse, _, _ = attend(z, z, z + 1, torch.zeros(2, 2, dtype=torch.bool), 1.0)
    assert torch.equal(O, z) and torch.isinf(lse).all()


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    q, k, v, dO = (torch.randn(s, generator=g, dtype=torch.float64)
                   for s in ((1, 2, 4, 5), (1, 1, 6, 5), (1, 1, 6, 5), (1, 2, 4, 5)))
    args = dict(window=3, sinks=1, scale=0.4)
    ref = window_reference(q, k, v, dO=dO, **args)
    h = 1e-5  # central differences: h^2 third derivatives, and 2^-53 / h
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for i in range(x.numel()):
            flat = x.view(-1)
            old = float(flat[i])
            loss = []
            for s in (h, -h):
                flat[i] = old + s
                loss.append(float((window_reference(q, k, v, **args)["o"] * dO).sum()))
            flat[i] = old
            assert abs((loss[0] - loss[1]) / (2 * h) - float(ref[name].view(-1)[i])) < 1e-7, (name, i)


@pytest.fixture(scope="module")
def lib():
    from attention_tiled_fwd_gb300 import build
    build.build()
    return nat.load()


A = 4096  # a fake, 16-byte aligned address: the call must be refused before it is touched
SIZES = dict(B=1, Hq=4, Hkv=2, Nq=8, Nk=16, kv_rows=16, D=64, window=4, sinks=1, scale=0.125, dtype=nat.FA_BF16,
             grad=nat.FA_F32)
BAD = [(dict(B=0), "SHAPE"), (dict(Hq=0), "SHAPE"), (dict(Hkv=0), "SHAPE"), (dict(Hkv=3), "SHAPE"), (dict(Nq=0), "SHAPE"),
       (dict(Nq=17), "SHAPE"), (dict(Nk=0), "SHAPE"), (dict(window=0), "SHAPE"), (dict(window=-1), "SHAPE"),
       (dict(sinks=-1), "SHAPE"), (dict(Nk=(1 << 29) + 1, kv_rows=(1 << 29) + 1), "SHAPE"),
       (dict(B=65535, Hq=65535, Hkv=65535, Nq=16), "SHAPE"), (dict(D=12), "HEAD_DIM"), (dict(D=264), "HEAD_DIM"),
       (dict(scale=0.0), "SCALE"), (dict(scale=-1.0), "SCALE"), (dict(scale=math.nan), "SCALE"),
       (dict(scale=math.inf), "SCALE"), (dict(scale=3e38), "SCALE"), (dict(dtype=nat.FA_F32), "DTYPE"), (dict(dtype=9), "DTYPE")]


def _err(name):
    return getattr(nat, "FA_ERR_" + name)


def _calls(lib, **kw):
    """Status of the forward, dQ, dK/dV and the whole backward with these arguments; pointers are fakes."""
    a = dict(SIZES, ptr=A)
    a.update(kw)
    p = a["ptr"]
    s = [a[n] for n in ("B", "Hq", "Hkv", "Nq", "Nk")]
    m = [a["D"], a["window"], a["sinks"], a["scale"], a["dtype"]]
    return (lib.fa_window_forward(p, A, A, A, A, *s, a["kv_rows"], *m, None),
            lib.fa_window_backward_dq(p, A, A, A, A, A, A, A, *s, *m, a["grad"], None),
            lib.fa_window_backward_dkdv(p, A, A, A, A, A, A, A, *s, *m, a["grad"], A, 1 << 30, None),
            lib.fa_window_backward(p, A, A, A, A, A, A, A, A, A, *s, *m, a["grad"], A, 1 << 30, None))


@pytest.mark.parametrize("kw,code", BAD)
def test_window_refusals(lib, kw, code):
    assert set(_calls(lib, **kw)) == {_err(code)}


def test_window_refusals_of_one_call(lib):
    assert _calls(lib, kv_rows=15)[0] == nat.FA_ERR_SHAPE
    assert _calls(lib, grad=7)[1:] == (nat.FA_ERR_DTYPE,) * 3
    assert set(_calls(lib, ptr=None)) == {nat.FA_ERR_NULL}
    assert set(_calls(lib, ptr=A + 8)) == {nat.FA_ERR_ALIGN}
    out = ctypes.c_size_t(0)
    assert lib.fa_window_backward_workspace_bytes(1, 4, 2, 8, 16, 64, 4, 1, None) == nat.FA_ERR_NULL
    assert lib.fa_window_backward_workspace_bytes(1, 4, 2, 8, 16, 64, 0, 1, ctypes.byref(out)) == nat.FA_ERR_SHAPE
    assert lib.fa_window_backward_workspace_bytes(1, 4, 2, 8, 16, 64, 4, 1, ctypes.byref(out)) == nat.FA_OK


@pytest.mark.parametrize("Hkv,N,sinks", [(8, 8192, 2560), (64, 32768, 4096), (512, 4096, 1), (1, 65536, 60000)])
def test_backward_workspace_stays_small(lib, Hkv, N, sinks):
    # partials of the sink tiles: at most four chunks an SM, beside two for each of less than four sink tiles an SM
    out = ctypes.c_size_t(0)
    for D in (64, 128, 256):
        assert lib.fa_window_backward_workspace_bytes(1, 4 * Hkv, Hkv, N, N, D, 256, sinks, ctypes.byref(out)) == nat.FA_OK
        assert out.value <= 12 * 160 * 2 * 4 * 128 * D


def _token(lib, **kw):
    a = dict(q=A, lens=A, B=2, Hq=4, Hkv=2, n_q=1, N=64, D=128, window=8, sinks=1, scale=0.1)
    a.update(kw)
    return lib.fa_window_decode(a["q"], A, A, a["lens"], A, A, *(a[n] for n in ("B", "Hq", "Hkv", "n_q", "N", "D", "window",
                                                                              "sinks", "scale")), A, 1 << 30, None)


def _prefix(lib, **kw):
    a = dict(q=A, lens=A, B=2, Hq=4, Hkv=2, n_q=1, P=100, N=64, D=128, scale=0.1, ws=A)
    a.update(kw)
    return lib.fa_prefix_decode(a["q"], A, A, A, A, a["lens"], A, A, *(a[n] for n in ("B", "Hq", "Hkv", "n_q", "P", "N", "D",
                                                                                    "scale")), a["ws"], 1 << 30, None)


@pytest.mark.parametrize("call", [_token, _prefix])
def test_decode_refusals(lib, call):
    for kw, code in ((dict(n_q=0), "SHAPE"), (dict(n_q=17), "SHAPE"), (dict(Hkv=3), "SHAPE"), (dict(N=0), "SHAPE"),
                     (dict(N=(1 << 29) + 1), "SHAPE"), (dict(B=65536), "SHAPE"), (dict(D=96), "HEAD_DIM"),
                     (dict(D=192), "HEAD_DIM"), (dict(scale=0.0), "SCALE"), (dict(scale=math.nan), "SCALE"),
                     (dict(q=None), "NULL"), (dict(q=A + 2), "ALIGN")):
        assert call(lib, **kw) == _err(code), kw


def test_decode_refusals_of_one_call(lib):
    assert _token(lib, window=0) == nat.FA_ERR_SHAPE
    assert _token(lib, sinks=-1) == nat.FA_ERR_SHAPE
    assert _token(lib, n_q=5, N=4) == nat.FA_ERR_SHAPE
    assert _prefix(lib, P=0) == nat.FA_ERR_SHAPE
    assert _prefix(lib, ws=None) == nat.FA_ERR_NULL
    out = ctypes.c_size_t(0)
    assert lib.fa_prefix_decode_workspace_bytes(2, 4, 2, 1, 100, 64, 128, None) == nat.FA_ERR_NULL
    assert lib.fa_window_decode_workspace_bytes(2, 4, 2, 1, 64, 128, 8, 1, None) == nat.FA_ERR_NULL
    assert lib.fa_prefix_decode_workspace_bytes(2, 4, 2, 1, 100, 64, 128, ctypes.byref(out)) == nat.FA_OK
    # at least one partial (O, m, l) of the prefix and one of the cache per row
    assert out.value >= 2 * 8 * 130 * 4


# ------------------------------------------------------------------ GPU
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# B, Hq, Hkv, Nq, Nk, D, window, sinks.
WINDOWS = [
    (1, 1, 1, 1, 1, 64, 1, 0), (1, 2, 1, 1, 300, 128, 7, 2), (2, 4, 2, 200, 200, 128, 128, 1),
    (1, 4, 1, 129, 1000, 64, 100, 0), (1, 2, 2, 77, 640, 128, 64, 130), (1, 3, 1, 300, 300, 80, 1000, 3),
    (2, 2, 1, 500, 777, 192, 130, 4), (1, 2, 2, 260, 260, 256, 90, 1), (1, 1, 1, 700, 700, 8, 33, 40),
    (4, 8, 4, 700, 700, 128, 200, 4), (4, 8, 8, 700, 700, 64, 300, 5), (4, 9, 3, 650, 801, 128, 129, 0),
    (3, 8, 8, 1001, 1001, 128, 256, 140), (2, 16, 4, 900, 1100, 64, 700, 1), (4, 8, 8, 600, 600, 128, 5000, 0),
    (3, 16, 2, 513, 2000, 40, 1, 0), (2, 16, 4, 800, 800, 256, 300, 20), (4, 8, 8, 640, 640, 96, 128, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", WINDOWS)
def test_window_forward(case):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, Nq, Nk, D, window, sinks = case
    g = _gen(sum(case))
    rows = Nk + 3
    q, k, v = _randn(g, B, Hq, Nq, D), _randn(g, B, Hkv, rows, D), _randn(g, B, Hkv, rows, D)
    # keys that no row sees: room behind the sequence, and what lies between the sinks and the first window
    first = Nk - Nq - window + 1
    ref = window_reference(q, k[:, :, :Nk], v[:, :, :Nk], window, sinks, 1 / math.sqrt(D))
    for t in (k, v):
        t[:, :, Nk:] = float("nan")
        if first > sinks:
            t[:, :, sinks:first] = float("nan")
    o, lse = fa.fa_window_forward(q, k, v, window, sinks, kv_len=Nk)
    assert fa.fa_device_status() == 0
    check(o, ref["o"], ref["o_bound"], "O")
    check_lse(lse, ref["lse"], "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", WINDOWS + [(1, 2, 1, 40, 900, 64, 50, 0), (1, 2, 1, 40, 900, 128, 50, 3),
                                            (1, 2, 1, 40, 900, 256, 50, 1), (1, 4, 2, 1500, 1500, 128, 64, 4), (1, 4, 2, 1500, 1500, 64, 64, 4),
                                            (2, 3, 1, 1700, 1800, 256, 60, 200), (1, 6, 2, 2000, 2000, 80, 100, 300),
                                            (1, 2, 2, 2000, 4000, 40, 30, 7), (1, 128, 32, 1999, 1999, 64, 64, 4),
                                            (2, 64, 64, 2000, 2100, 40, 60, 16)])
def test_window_backward(case, grad_dtype):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, Nq, Nk, D, window, sinks = case
    g = _gen(1 + sum(case))
    q, k, v, dO = (_randn(g, B, h, n, D) for h, n in ((Hq, Nq), (Hkv, Nk), (Hkv, Nk), (Hq, Nq)))
    ref = window_reference(q, k, v, window, sinks, 0.11, dO)
    o, lse = fa.fa_window_forward(q, k, v, window, sinks, scale=0.11)
    kw = dict(scale=0.11, grad_dtype=grad_dtype)
    dq, delta = fa.fa_window_backward_dq(q, k, v, o, dO, lse, window, sinks, **kw)
    # the outputs and the workspace hold NaN before the call: nothing relies on what was there
    need = fa.fa_window_backward_workspace_bytes(B, Hq, Hkv, Nq, Nk, D, window, sinks)
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    dk, dv = (torch.full(k.shape, float("nan"), dtype=grad_dtype, device="cuda") for _ in range(2))
    fa.fa_window_backward_dkdv(q, k, v, dO, lse, delta, window, sinks, dk=dk, dv=dv, workspace=ws, **kw)
    assert fa.fa_device_status() == 0
    check(delta, ref["delta"], ref["delta_bound"], "delta")
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        stored = U * ref[name].abs() if grad_dtype == torch.bfloat16 else 0.0
        check(t, ref[name], ref[name + "_bound"] + stored, name)
    first = Nk - Nq - window + 1
    if first > sinks:
        assert not dk[:, :, sinks:first].any() and not dv[:, :, sinks:first].any()
    # again, and both halves in one call: the same bits
    again = fa.fa_window_backward_dkdv(q, k, v, dO, lse, delta, window, sinks, **kw)
    assert torch.equal(again[0], dk) and torch.equal(again[1], dv)
    for a, b in zip(fa.fa_window_backward(q, k, v, o, dO, lse, window, sinks, **kw), (dq, dk, dv, delta)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_window_attention_autograd():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(5)
    # a transposed projection: [B, N, H, D] seen as [B, H, N, D]
    q = _randn(g, 2, 300, 4, 64).transpose(1, 2).requires_grad_()
    k, v = (_randn(g, 2, 300, 2, 64).transpose(1, 2).requires_grad_() for _ in range(2))
    dO = _randn(g, 2, 4, 300, 64)
    o = fa.window_attention(q, k, v, 50, 2)
    dq, dk, dv = torch.autograd.grad(o, (q, k, v), dO)
    ref = window_reference(q.detach(), k.detach(), v.detach(), 50, 2, 1 / 8, dO)
    check(o.detach(), ref["o"], ref["o_bound"], "O")
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        check(t, ref[name], ref[name + "_bound"] + U * ref[name].abs(), name)
    # a gradient of one input alone
    (only,) = torch.autograd.grad(fa.window_attention(q, k.detach(), v.detach(), 50, 2), (q,), dO)
    assert torch.equal(only, dq)


@pytest.mark.gpu
def test_window_covering_everything_is_causal_attention():
    """One head per key head and a window of the whole sequence: fa_forward's causal results, within two bounds."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(6)
    q, k, v = (_randn(g, 1, 2, 500, 128) for _ in range(3))
    ref = window_reference(q, k, v, 500, 0, 1 / math.sqrt(128))
    for o, lse in (fa.fa_forward(q, k, v, causal=True), fa.fa_window_forward(q, k, v, 1 << 40),
                   fa.fa_window_forward(q, k, v, 500, 77)):
        check(o, ref["o"], ref["o_bound"], "O")
        check_lse(lse, ref["lse"], "LSE")


# B, Hq, Hkv, n_q, N, D, window, sinks, lens
TOKENS = [
    (1, 1, 1, 1, 1, 64, 1, 0, [1]), (3, 4, 2, 1, 500, 128, 100, 4, [0, 1, 500]), (2, 8, 1, 3, 777, 128, 64, 1, [2, 777]),
    (1, 16, 4, 1, 5000, 128, 1024, 4, [4001]), (4, 2, 2, 16, 300, 64, 40, 0, [300, 15, 16, 200]),
    (2, 16, 1, 8, 1000, 256, 500, 130, [999, 64]), (1, 2, 1, 2, 9000, 64, 9000, 0, [8191]), (2, 3, 3, 5, 90, 256, 1, 1, [90, 33]),
    (40, 32, 8, 1, 300, 128, 64, 2, None), (5, 6, 2, 4, 2500, 128, 200, 70, [2500, 100, 264, 265, 3]),
    (1, 4, 4, 1, 30000, 256, 30000, 0, [29999]), (2, 20, 1, 1, 640, 64, 128, 64, [640, 320]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", TOKENS)
def test_window_decode(case):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, n_q, N, D, window, sinks, lens = case
    g = _gen(N + D)
    q, k, v = _randn(g, B, Hq, n_q, D), _randn(g, B, Hkv, N, D), _randn(g, B, Hkv, N, D)
    ln = torch.tensor([N] * B if lens is None else lens, dtype=torch.int32, device="cuda")
    ref = cached_reference(q, k, v, ln.tolist(), window, sinks, 1 / math.sqrt(D))
    for b, n in enumerate(ln.tolist()):
        for t in (k, v):  # what no row sees
            t[b, :, n:] = float("nan")
            lo = max(0, n - n_q) - window + 1
            if lo > sinks:
                t[b, :, sinks:lo] = float("inf")
    need = fa.fa_window_decode_workspace_bytes(B, Hq, Hkv, n_q, N, D, window, sinks)
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    o, lse = fa.fa_window_decode(q, k, v, window, sinks, lens=None if lens is None else ln, workspace=ws)
    assert fa.fa_device_status() == 0
    check(o, ref["o"], ref["o_bound"], "O")
    check_lse(lse, ref["lse"], "LSE")
    again = fa.fa_window_decode(q, k, v, window, sinks, lens=None if lens is None else ln)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


# B, Hq, Hkv, n_q, P, N, D, lens
PREFIXES = [
    (1, 1, 1, 1, 1, 1, 64, [1]), (5, 16, 4, 1, 777, 128, 128, [1, 100, 37, 0, 128]), (3, 4, 1, 3, 1000, 64, 64, [3, 2, 64]),
    (40, 8, 2, 1, 513, 40, 128, None), (2, 16, 1, 16, 700, 50, 128, [50, 7]), (3, 16, 1, 16, 300, 200, 256, [16, 0, 200]),
    (7, 6, 2, 2, 3000, 300, 256, [2, 300, 5, 64, 65, 0, 1]), (130, 4, 4, 1, 260, 9, 64, None),
    (2, 40, 1, 4, 400, 30, 64, [30, 4]), (33, 5, 5, 1, 20000, 16, 128, None), (1, 2, 1, 1, 128, 4000, 128, [3333]),
    (300, 4, 4, 1, 260, 9, 64, None), (140, 16, 2, 1, 300, 20, 256, None), (90, 16, 1, 1, 1500, 700, 128, None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", PREFIXES)
def test_prefix_decode(case):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, n_q, P, N, D, lens = case
    g = _gen(P + N)
    q, k, v = _randn(g, B, Hq, n_q, D), _randn(g, B, Hkv, N, D), _randn(g, B, Hkv, N, D)
    kp, vp = _randn(g, Hkv, P, D), _randn(g, Hkv, P, D)
    ln = torch.tensor([N] * B if lens is None else lens, dtype=torch.int32, device="cuda")
    ref = cached_reference(q, k, v, ln.tolist(), N, 0, 1 / math.sqrt(D), kp, vp)
    for b, n in enumerate(ln.tolist()):
        k[b, :, n:] = float("nan")
        v[b, :, n:] = float("nan")
    need = fa.fa_prefix_decode_workspace_bytes(B, Hq, Hkv, n_q, P, N, D)
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    o, lse = fa.fa_prefix_decode(q, kp, vp, k, v, lens=None if lens is None else ln, workspace=ws)
    assert fa.fa_device_status() == 0
    check(o, ref["o"], ref["o_bound"], "O")
    check_lse(lse, ref["lse"], "LSE")
    again = fa.fa_prefix_decode(q, kp, vp, k, v, lens=None if lens is None else ln)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.gpu
def test_lens_outside_the_cache_are_clamped():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(9)
    q, k, v = _randn(g, 3, 2, 1, 64), _randn(g, 3, 2, 70, 64), _randn(g, 3, 2, 70, 64)
    for bad, good in (([-5, 71, 1 << 30], [0, 70, 70]),):
        a, b = (fa.fa_window_decode(q, k, v, 20, 2, lens=torch.tensor(x, dtype=torch.int32, device="cuda")) for x in (bad, good))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert not a[0][0].any() and torch.isinf(a[1][0]).all()


@pytest.mark.gpu
def test_prefill_in_chunks_then_tokens_then_samples():
    """A prompt prefilled in two chunks into a cache, tokens decoded one and three at a time, and the same rows as a
    batch of samples behind the prompt as a shared prefix: every route gives the rows of one whole forward."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(11)
    Hq, Hkv, N, D, W, S = 8, 2, 400, 128, 96, 4
    q, k, v = _randn(g, 1, Hq, N, D), _randn(g, 1, Hkv, N, D), _randn(g, 1, Hkv, N, D)
    ref = window_reference(q, k, v, W, S, 1 / math.sqrt(D))
    cache = [torch.full((1, Hkv, 512, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def rows(o, lse, r0, r1):
        check(o, ref["o"][:, :, r0:r1], ref["o_bound"][:, :, r0:r1], f"O {r0}..{r1}")
        check_lse(lse, ref["lse"][:, :, r0:r1], f"LSE {r0}..{r1}")

    for r0, r1 in ((0, 150), (150, 390)):
        for c, t in zip(cache, (k, v)):
            c[:, :, r0:r1] = t[:, :, r0:r1]
        rows(*fa.fa_window_forward(q[:, :, r0:r1].contiguous(), *cache, W, S, kv_len=r1), r0, r1)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    for r0, r1 in ((390, 391), (391, 394), (394, 400)):
        for c, t in zip(cache, (k, v)):
            c[:, :, r0:r1] = t[:, :, r0:r1]
        lens.fill_(r1)
        rows(*fa.fa_window_decode(q[:, :, r0:r1].contiguous(), *cache, W, S, lens=lens), r0, r1)
    # samples: every sequence's own cache holds a different number of the last keys behind the same prompt
    full = window_reference(q, k, v, N, 0, 1 / math.sqrt(D))
    kp, vp = (t[0, :, :380].contiguous() for t in (k, v))
    own_k, own_v = (t[:, :, 380:].expand(3, -1, -1, -1).contiguous() for t in (k, v))
    lens = torch.tensor([3, 20, 9], dtype=torch.int32, device="cuda")
    qs = torch.cat([q[:, :, 379 + n:380 + n] for n in lens.tolist()]).contiguous()
    o, lse = fa.fa_prefix_decode(qs, kp, vp, own_k, own_v, lens=lens)
    for b, n in enumerate(lens.tolist()):
        check(o[b], full["o"][0, :, 379 + n:380 + n], full["o_bound"][0, :, 379 + n:380 + n], f"sample {b}")
        check_lse(lse[b], full["lse"][0, :, 379 + n:380 + n], f"sample {b}")


@pytest.mark.gpu
def test_captured_calls_follow_their_inputs():
    """A captured graph of both decodes and a training step's kernels, replayed with new values in the same buffers."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(13)
    q, k, v, dO = (_randn(g, 2, h, 300, 64) for h in (4, 2, 2, 4))
    kp, vp = _randn(g, 2, 200, 64), _randn(g, 2, 200, 64)
    lens = torch.tensor([300, 17], dtype=torch.int32, device="cuda")
    qt = q[:, :, :1].contiguous()

    def work():
        o, lse = fa.fa_window_forward(q, k, v, 40, 2)
        dq, delta = fa.fa_window_backward_dq(q, k, v, o, dO, lse, 40, 2)
        return (o, lse, dq, *fa.fa_window_backward_dkdv(q, k, v, dO, lse, delta, 40, 2),
                *fa.fa_window_decode(qt, k, v, 40, 2, lens=lens), *fa.fa_prefix_decode(qt, kp, vp, k, v, lens=lens))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for step in range(2):
        for t in (q, k, v, dO, kp, vp):
            t.copy_(_randn(g, *t.shape))
        lens.copy_(torch.tensor([step, 299], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, work()):
            assert torch.equal(a, b)
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
def test_side_stream_without_a_current_stream_switch():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(15)
    q, k, v = _randn(g, 2, 4, 1, 128), _randn(g, 2, 2, 3000, 128), _randn(g, 2, 2, 3000, 128)
    want = fa.fa_window_decode(q, k, v, 2500, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [fa.fa_window_decode(q, k, v, 2500, 2, stream=side) for _ in range(4)]
    side.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_binding_refusals():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(17)
    q, k = _randn(g, 1, 4, 8, 64), _randn(g, 1, 2, 16, 64)
    ok = fa.fa_window_forward(q, k, k, 4)
    assert ok[0].shape == q.shape
    with pytest.raises(ValueError):
        fa.fa_window_forward(q, _randn(g, 1, 3, 16, 64), _randn(g, 1, 3, 16, 64), 4)   # 4 heads over 3
    with pytest.raises(ValueError):
        fa.fa_window_forward(q, k, k[:, :, :8], 4)                                     # v is not k's shape
    with pytest.raises(ValueError):
        fa.fa_window_forward(q.transpose(2, 3).contiguous().transpose(2, 3), k, k, 4)  # not contiguous
    with pytest.raises(ValueError):
        fa.fa_window_forward(q.cpu(), k, k, 4)
    with pytest.raises(TypeError):
        fa.fa_window_forward(q.half(), k.half(), k.half(), 4)
    with pytest.raises(fa.FAError) as e:
        fa.fa_window_forward(q, k, k, 4, kv_len=17)
    assert e.value.code == nat.FA_ERR_SHAPE
    with pytest.raises(TypeError):
        fa.fa_window_decode(q, k, k, 4, lens=torch.tensor([16], device="cuda"))        # int64
    with pytest.raises(ValueError):
        fa.fa_window_decode(q, k, k, 4, lens=torch.tensor([16, 3], dtype=torch.int32, device="cuda"))
    big = _randn(g, 1, 2, 5000, 64)
    with pytest.raises(fa.FAError) as e:
        fa.fa_window_decode(q, big, big, 5000, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == nat.FA_ERR_WORKSPACE
    with pytest.raises(fa.FAError) as e:
        fa.fa_prefix_decode(q, big[0], big[0], k, k, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == nat.FA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        fa.fa_prefix_decode(q, big, big, k, k)                                         # a prefix has no batch


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Nq,window,sinks", [(300, 70, 0), (300, 70, 3), (300, 500, 0), (20, 9, 0), (200, 40, 50)])
def test_a_nan_shows_where_it_is_seen_and_nowhere_else(D, Nq, window, sinks):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(D + Nq)
    q, k, v = (_randn(g, 1, 2, Nq, D) for _ in range(3))
    ref = window_reference(q, k, v, window, sinks, 1 / math.sqrt(D))
    seen = visible(torch.arange(Nq, device="cuda"), Nq, window, sinks)
    for head, key, row, value in ((0, Nq // 2, Nq // 3, "nan"), (1, 0, Nq - 1, "inf")):
        kk, qq = k.clone(), q.clone()
        kk[0, head, key] = float("nan")
        qq[0, head, row] = float(value)  # an infinite q makes scores of +-inf and NaN: its row is NaN
        bad = torch.zeros(2, Nq, dtype=torch.bool, device="cuda")
        bad[head] = seen[:, key]
        bad[head, row] = True
        o, lse = fa.fa_window_forward(qq, kk, v, window, sinks)
        assert torch.equal(torch.isnan(lse[0]), bad)
        assert torch.isnan(o[0][bad]).all()
        check(o[0][~bad], ref["o"][0][~bad], ref["o_bound"][0][~bad], "O")


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,P", [(40, 60), (5000, 3000), (64, 20000)])
def test_a_nan_shows_in_the_decodes(D, N, P):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(D + N)
    B, Hq, Hkv = 3, 4, 2
    q, k, v = _randn(g, B, Hq, 1, D), _randn(g, B, Hkv, N, D), _randn(g, B, Hkv, N, D)
    kp, vp = _randn(g, Hkv, P, D), _randn(g, Hkv, P, D)
    lens = torch.tensor([N, 0, N // 2], dtype=torch.int32, device="cuda")
    q[0, 1] = float("nan")            # every score of a row
    k[2, 0, N // 2 - 1] = float("nan")  # the newest key of a sequence
    k[2, 1, N // 2] = float("nan")      # a key that nothing sees
    bad = torch.zeros(B, Hq, dtype=torch.bool, device="cuda")
    bad[0, 1], bad[2, 0], bad[2, 1] = True, True, True
    for call in (lambda: fa.fa_window_decode(q, k, v, 7, 1, lens=lens), lambda: fa.fa_window_decode(q, k, v, N, 0, lens=lens),
                 lambda: fa.fa_prefix_decode(q, kp, vp, k, v, lens=lens)):
        o, lse = call()
        assert torch.equal(torch.isnan(lse[..., 0]), bad)
        assert torch.equal(torch.isnan(o[:, :, 0]).all(-1), bad) and torch.equal(torch.isnan(o[:, :, 0]).any(-1), bad)
    kp[1, P - 1] = float("nan")         # the prefix's last key, for one key head
    bad[:, 2:] = True
    o, lse = fa.fa_prefix_decode(q, kp, vp, k, v, lens=lens)
    assert torch.equal(torch.isnan(lse[..., 0]), bad) and torch.equal(torch.isnan(o[:, :, 0]).all(-1), bad)


@pytest.mark.gpu
def test_second_derivatives_are_refused():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    q = _randn(_gen(1), 1, 1, 40, 64).requires_grad_()
    o = fa.window_attention(q, q, q, 9)
    with pytest.raises(RuntimeError, match="create_graph"):
        torch.autograd.grad(o.float().square().sum(), q, create_graph=True)


@pytest.mark.gpu
def test_two_streams_at_once():
    """The same calls from two streams, each with workspaces of its own, give what they give one after the other."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(11)
    q, k, v = _randn(g, 2, 8, 900, 128), _randn(g, 2, 2, 900, 128), _randn(g, 2, 2, 900, 128)
    dO = _randn(g, 2, 8, 900, 128)
    tq, kp, vp = _randn(g, 2, 8, 1, 128), _randn(g, 2, 5000, 128), _randn(g, 2, 5000, 128)

    def calls(stream):
        o, lse = fa.fa_window_forward(q, k, v, 100, 5, stream=stream)
        grads = fa.fa_window_backward(q, k, v, o, dO, lse, 100, 5, stream=stream)
        return (o, lse, *grads, *fa.fa_window_decode(tq, k, v, 900, 0, stream=stream),
                *fa.fa_prefix_decode(tq, kp, vp, k, v, stream=stream))

    expect = calls(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [calls(s) for _ in range(20) for s in streams]
    torch.cuda.synchronize()
    assert fa.fa_device_status() == 0
    for outs in got:
        for a, b in zip(outs, expect):
            assert torch.equal(a, b)


def _room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB of free device memory")


@pytest.mark.gpu
def test_caches_beyond_32_bit_offsets():
    """A sequence at the end of a cache of more than 2^32 elements; what its rows do not see is left unwritten."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    _room(20)
    g = _gen(12)
    N, D, window, sinks = (1 << 24) + 77, 256, 100, 3
    k, v = (torch.empty(1, 1, N, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = [_randn(g, 1, 1, 203, D) for _ in range(2)]
    for big, s in zip((k, v), small):  # rows 0 .. 2 and the last 200
        big[:, :, :3] = s[:, :, :3]
        big[:, :, N - 200:] = s[:, :, 3:]
    q = _randn(g, 1, 2, 16, D)
    ref = window_reference(q, *small, window, sinks, 1 / math.sqrt(D))
    for o, lse in (fa.fa_window_decode(q, k, v, window, sinks), fa.fa_window_forward(q, k, v, window, sinks)):
        check(o, ref["o"], ref["o_bound"], "O")
        check_lse(lse, ref["lse"], "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_heads_beyond_32_bit_offsets(D):
    """The last head of tensors of more than 2^32 elements, forward and backward, is what it is by itself."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    _room(90)
    g = _gen(13)
    H, N, window = 8, (1 << 32) // (8 * D) + 1000, 70
    q, k, v, dO = (torch.zeros(1, H, N, D, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    for t in (q, k, v, dO):
        t[:, -1] = _randn(g, 1, N, D)
    last = [t[:, -1:].contiguous() for t in (q, k, v, dO)]
    o, lse = fa.fa_window_forward(q, k, v, window)
    o1, lse1 = fa.fa_window_forward(*last[:3], window)
    assert torch.equal(o[:, -1:], o1) and torch.equal(lse[:, -1:], lse1)
    dq, dk, dv, delta = fa.fa_window_backward(q, k, v, o, dO, lse, window, grad_dtype=torch.bfloat16)
    alone = fa.fa_window_backward(*last[:3], o1, last[3], lse1, window, grad_dtype=torch.bfloat16)
    for a, b in zip((dq, dk, dv, delta), alone):
        assert torch.equal(a[:, -1:], b)


@pytest.mark.gpu
def test_gradients_of_broadcast_and_strided_inputs():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(14)
    B, H, N, D = 3, 4, 150, 64
    q = _randn(g, B, N, H, D).requires_grad_()        # heads behind rows: a strided view
    kv = _randn(g, 1, 1, N, D).requires_grad_()       # one tensor for keys and values of every sequence
    dO = _randn(g, B, H, N, D)
    k = kv.expand(B, 1, N, D)
    o = fa.window_attention(q.transpose(1, 2), k, k, 40, 2)
    dq, dkv = torch.autograd.grad(o, (q, kv), dO)
    ref = window_reference(q.detach().transpose(1, 2), k.detach(), k.detach(), 40, 2, 1 / math.sqrt(D), dO)
    check(dq.transpose(1, 2), ref["dq"], ref["dq_bound"] + U * ref["dq"].abs(), "dq")
    # three sequences' dK and dV, each rounded to bf16, added by autograd in two sums that each round once more: at most
    # (2 + 3) half steps of the magnitudes that are added
    parts = [ref[n].abs() for n in ("dk", "dv")]
    bound = (ref["dk_bound"] + ref["dv_bound"]).sum(0, keepdim=True) + 5 * U * (parts[0] + parts[1]).sum(0, keepdim=True)
    check(dkv, (ref["dk"] + ref["dv"]).sum(0, keepdim=True), bound, "dk + dv")


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(2, 6, 2, 300, 300, 64, 40, 3), (1, 4, 4, 90, 90, 128, 500, 0), (1, 3, 1, 200, 260, 80, 33, 0),
                                  (1, 2, 1, 130, 257, 256, 9, 140), (2, 2, 2, 150, 278, 192, 64, 1), (1, 1, 1, 1, 1, 128, 1, 0),
                                  (2, 2, 2, 150, 277, 192, 64, 1)])
def test_delta_of_the_first_rows_does_not_carry_o_rounding(case):
    """Rows at positions below 128: delta = sum P dP.  P is off by 2^-11 of its value (its score and its row's LSE), the
    rest is fp32, so delta by 2^-10 sum P |dP|; with the stored O it would be up to 2^-8 sum |dO O|."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, Nq, Nk, D, window, sinks = case
    g = _gen(sum(case))
    q, k, v, dO = (_randn(g, B, h, n, D) for h, n in ((Hq, Nq), (Hkv, Nk), (Hkv, Nk), (Hq, Nq)))
    o, lse = fa.fa_window_forward(q, k, v, window, sinks)
    _, delta = fa.fa_window_backward_dq(q, k, v, o, dO, lse, window, sinks)
    G, off = Hq // Hkv, Nk - Nq
    kk, vv = (t.double().repeat_interleave(G, 1) for t in (k, v))
    pos = torch.arange(off, Nk, device="cuda")
    _, _, P, _ = attend(q.double(), kk, vv, visible(pos, Nk, window, sinks), 1 / math.sqrt(D))
    dP = torch.matmul(dO.double(), vv.transpose(-1, -2))
    early = pos < 128
    assert early.any() == (off < 128)
    if off < 128:
        check(delta[:, :, early], (P * dP).sum(-1)[:, :, early], 2.0 ** -10 * (P * dP.abs()).sum(-1)[:, :, early], "delta")
