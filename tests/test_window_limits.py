"""Windowed and shared-prefix calls at the limits of their contracts: workspaces at every alignment that is allowed,
sizes past the C interface's integers, calls whose single steps are short but whose waits are not."""
import ctypes

import pytest
import torch

from attention_tiled_fwd_gb300 import _native as nat
from helpers import cuda_or_skip


@pytest.fixture(scope="module")
def lib():
    from attention_tiled_fwd_gb300 import build
    build.build()
    return nat.load()


# ------------------------------------------------------------------ the prefix's partials are stored 32 bytes at a time
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_workspace_has_room_to_align(lib, D):
    # one row, one prefix key, one cache key: one 128-row partial of O (fp32), m and l, and nothing of the cache.  A
    # workspace at 16 mod 32 loses 16 bytes before the first 32-byte boundary.
    out = ctypes.c_size_t(0)
    assert lib.fa_prefix_decode_workspace_bytes(1, 1, 1, 1, 1, 1, D, ctypes.byref(out)) == nat.FA_OK
    assert out.value >= 128 * (D * 4 + 8) + 16


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(3, 8, 2, 1, 300, 40, 64), (70, 16, 4, 2, 900, 1200, 128), (5, 4, 1, 3, 400, 70, 256),
                                  (140, 16, 2, 1, 300, 20, 256)])
def test_prefix_workspace_at_16_mod_32(case):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, n_q, P, N, D = case
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(case))
    q, k, v = _randn(g, B, Hq, n_q, D), _randn(g, B, Hkv, N, D), _randn(g, B, Hkv, N, D)
    kp, vp = _randn(g, Hkv, P, D), _randn(g, Hkv, P, D)
    need = fa.fa_prefix_decode_workspace_bytes(B, Hq, Hkv, n_q, P, N, D)
    want = fa.fa_prefix_decode(q, kp, vp, k, v)
    buf = torch.empty(need + 96, dtype=torch.uint8, device="cuda")
    base = -buf.data_ptr() % 32
    for at in (base, base + 16):  # at 0 and at 16 mod 32, of exactly the size that the query gives
        buf.fill_(0xA5)
        ws = buf[at:at + need]
        assert ws.data_ptr() % 32 == at - base
        got = fa.fa_prefix_decode(q, kp, vp, k, v, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (buf[:at] == 0xA5).all() and (buf[at + need:] == 0xA5).all()
    assert fa.fa_device_status() == 0
    with pytest.raises(fa.FAError) as e:
        fa.fa_prefix_decode(q, kp, vp, k, v, workspace=buf[base + 16:base + need - 16])
    assert e.value.code == nat.FA_ERR_WORKSPACE


# ------------------------------------------------------------------ sizes are C ints: a longer one must not wrap around
def test_size_queries_refuse_what_is_no_c_int(lib):
    import attention_tiled_fwd_gb300 as fa
    calls = ((fa.fa_window_backward_workspace_bytes, [1, 4, 2, 8, 16, 64, 4, 1], 6),  # (window and sinks saturate)
             (fa.fa_window_decode_workspace_bytes, [1, 4, 2, 1, 64, 64, 4, 1], 6),
             (fa.fa_prefix_decode_workspace_bytes, [1, 4, 2, 1, 100, 64, 64], 7))
    for call, sizes, n in calls:
        call(*sizes)
        for i in range(n):
            for wrong in (sizes[i] + (1 << 32), sizes[i] - (1 << 32)):
                with pytest.raises(fa.FAError) as e:
                    call(*sizes[:i], wrong, *sizes[i + 1:])
                assert e.value.code == nat.FA_ERR_SHAPE


def test_calls_refuse_sizes_that_are_no_c_int(lib):
    """Refused before anything else of the tensors is looked at: these have no memory."""
    import attention_tiled_fwd_gb300 as fa

    def t(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="meta")

    q, k, kp = t(1, 4, 1, 64), t(1, 2, 16, 64), t(2, 16, 64)
    long = (1 << 32) + 16
    for call in (lambda: fa.fa_window_forward(q, k, k, 4, kv_len=long), lambda: fa.fa_window_forward(q, k, k, 4, kv_len=16 - (1 << 32)),
                 lambda: fa.fa_window_forward(t(1, 4, long, 8), t(1, 2, long, 8), t(1, 2, long, 8), 4),
                 lambda: fa.fa_window_forward(q, t(1, 2, long, 64), t(1, 2, long, 64), 4, kv_len=16),
                 lambda: fa.window_attention(t(long, 4, 8, 8), t(long, 4, 8, 8), t(long, 4, 8, 8), 4),
                 lambda: fa.fa_window_decode(q, t(1, 2, long, 64), t(1, 2, long, 64), 4),
                 lambda: fa.fa_prefix_decode(q, t(2, long, 64), t(2, long, 64), k, k),
                 lambda: fa.fa_prefix_decode(q, kp, kp, t(1, 2, long, 64), t(1, 2, long, 64))):
        with pytest.raises(fa.FAError) as e:
            call()
        assert e.value.code == nat.FA_ERR_SHAPE


# ------------------------------------------------------------------ no accumulator sums more than 2^21 products
MOST = 1 << 21
A = 4096  # a fake address: what passes the checks of sizes is refused as no device memory


def _statuses(lib, B, Hq, Hkv, Nq, Nk, D, window, sinks):
    """The forward's, dQ's, dK/dV's, the whole backward's and the size query's."""
    s, m = (B, Hq, Hkv, Nq, Nk), (D, window, sinks, 0.1, nat.FA_BF16)
    out = ctypes.c_size_t(0)
    return (lib.fa_window_forward(A, A, A, A, A, *s, Nk, *m, None),
            lib.fa_window_backward_dq(A, A, A, A, A, A, A, A, *s, *m, nat.FA_F32, None),
            lib.fa_window_backward_dkdv(A, A, A, A, A, A, A, A, *s, *m, nat.FA_F32, A, 1 << 40, None),
            lib.fa_window_backward(A, A, A, A, A, A, A, A, A, A, *s, *m, nat.FA_F32, A, 1 << 40, None),
            lib.fa_window_backward_workspace_bytes(*s, D, window, sinks, ctypes.byref(out)))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_sums_that_are_too_long_are_refused(lib, D):
    bad, passed = nat.FA_ERR_SHAPE, nat.FA_ERR_DEVICE_PTR
    # keys that a row sees
    assert _statuses(lib, 1, 1, 1, 128, MOST + 1, D, MOST + 1, 0) == (bad,) * 5
    assert _statuses(lib, 1, 1, 1, 128, 1 << 29, D, MOST - 3, 4) == (bad,) * 5
    assert _statuses(lib, 1, 1, 1, 128, 1 << 29, D, 4, (1 << 31) - 1) == (bad,) * 5
    assert _statuses(lib, 1, 1, 1, 128, 1 << 29, D, MOST - 4, 4) == (passed,) * 4 + (nat.FA_OK,)
    assert _statuses(lib, 1, 1, 1, 128, MOST, D, (1 << 31) - 1, 0) == (passed,) * 4 + (nat.FA_OK,)
    # rows of a group that see a key in their window
    assert _statuses(lib, 1, 16, 2, MOST // 8 + 1, MOST // 8 + 1, D, MOST // 8 + 1, 0) == (passed,) + (bad,) * 4
    assert _statuses(lib, 1, 16, 2, MOST // 8, MOST // 8, D, MOST, 0) == (passed,) * 4 + (nat.FA_OK,)


@pytest.mark.parametrize("D,Hq,Hkv,N,window,sinks", [(128, 8, 1, 1 << 22, 1 << 17, 4), (64, 8, 1, 1 << 22, 1 << 17, 40),
                                                     (256, 4, 2, 1 << 23, 1 << 18, 1), (256, 64, 1, 1 << 17, 64, 1 << 17)])
def test_rows_behind_the_sinks_are_cut_to_what_a_sum_holds(lib, D, Hq, Hkv, N, window, sinks):
    # partials: 1 + chunks of 128 x D floats for dK and dV of every sink tile; a chunk has 2^21 rows at most
    out = ctypes.c_size_t(0)
    assert lib.fa_window_backward_workspace_bytes(1, Hq, Hkv, N, N, D, window, sinks, ctypes.byref(out)) == nat.FA_OK
    rest = Hq // Hkv * (N - 127 - window)
    tiles = -(-sinks // 128)
    chunks = out.value // (8 * 128 * D * Hkv * tiles) - 1
    assert chunks * MOST >= rest


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_row_that_sees_the_most_keys(D):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    q = torch.zeros(1, 1, 3, D, dtype=torch.bfloat16, device="cuda")  # all scores are 0: O is the mean of v
    k, v = _randn(g, 1, 1, MOST, D), (0.3 * torch.randn(1, 1, MOST, D, generator=g, device="cuda") + 1).bfloat16()
    want = (v[0, 0].double().sum(0, keepdim=True) - torch.cat((v[0, 0, -2:].double().flip(0).cumsum(0).flip(0),
                                                                torch.zeros(1, D, dtype=torch.float64, device="cuda"))))
    seen = torch.arange(MOST - 2, MOST + 1, dtype=torch.float64, device="cuda")
    want /= seen[:, None]
    o, lse = fa.fa_window_forward(q, k, v, MOST)
    assert fa.fa_device_status() == 0
    # each of 2^21 addends loses less than 2^-25 of the sum so far, half of the final one on average: 2^-5 of the mean of
    # |v| (below 1.1), beside the roundings of P (exact here) and O (2^-8)
    assert ((o[0, 0].double() - want).abs() <= 1.1 * 2.0 ** -5 + 2.0 ** -8 * want).all()
    assert ((lse[0, 0].double() - torch.log(seen)).abs() <= 2.0 ** -12).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_token_splits_of_many_rows_and_long_caches(lib, D):
    # 128 heads of 16 rows on one key head fill the GPU with few splits; a warp adds up a quarter of a split's keys
    out = ctypes.c_size_t(0)
    rows, N = 128 * 16, 1 << 28
    assert lib.fa_window_decode_workspace_bytes(1, 128, 1, 16, N, D, N, 0, ctypes.byref(out)) == nat.FA_OK
    assert out.value // (rows * (D * 4 + 8)) * 4 * MOST >= N


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_chunks_of_a_long_prefix(lib, D):
    # 65535 rows of one key head fill the GPU uncut: 512 tiles of 128 rows, whose partials need D floats, m and l a chunk
    out = ctypes.c_size_t(0)
    P = 1 << 29
    assert lib.fa_prefix_decode_workspace_bytes(65535, 1, 1, 1, P, 1, D, ctypes.byref(out)) == nat.FA_OK
    assert out.value >= P // MOST * 512 * 128 * (D * 4 + 8)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_behind_a_long_prefix(D):
    """Scores of 0: O is the mean of v over the prefix and the own key, chunk by chunk within a sum of 2^21 keys."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    _room(30)
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    B, P = 40000, 4 * MOST + 77
    q = torch.zeros(B, 1, 1, D, dtype=torch.bfloat16, device="cuda")
    kp, vp = torch.zeros(1, P, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, P, D, dtype=torch.bfloat16, device="cuda")
    for c in range(0, P, MOST):
        vp[:, c:c + MOST] = (0.3 * torch.randn(1, min(MOST, P - c), D, generator=g, device="cuda") + 1).bfloat16()
    k, v = _randn(g, B, 1, 1, D), _randn(g, B, 1, 1, D)
    total = sum(vp[0, c:c + MOST].double().sum(0) for c in range(0, P, MOST))
    want = (total + v[:, 0, 0].double()) / (P + 1)
    o, lse = fa.fa_prefix_decode(q, kp, vp, k, v)
    assert fa.fa_device_status() == 0
    # as for a row that sees the most keys: 2^-5 of the mean of |v| (below 1.1), and O's rounding
    assert ((o[:, 0, 0].double() - want).abs() <= 1.1 * 2.0 ** -5 + 2.0 ** -8 * want.abs()).all()
    assert ((lse.double() - torch.log(torch.tensor(P + 1.0, dtype=torch.float64))).abs() <= 2.0 ** -12).all()


def _room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB of free device memory")


@pytest.mark.gpu
def test_a_step_that_the_backward_refuses_is_refused_at_once():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    N = MOST // 8 + 1
    q, k = (torch.zeros(1, h, N, 8, dtype=torch.bfloat16, device="cuda") for h in (8, 1))
    assert fa.window_attention(q, k, k, N).shape == q.shape  # a forward alone
    with pytest.raises(fa.FAError) as e:
        fa.window_attention(q.requires_grad_(), k, k, N)
    assert e.value.code == nat.FA_ERR_SHAPE
    assert fa.window_attention(q, k, k, N - 1).requires_grad
