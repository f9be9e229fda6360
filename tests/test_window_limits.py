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


# ------------------------------------------------------------------ waits inside a kernel are bounded by 1.5 s a step
# The longest window: every key step takes about a microsecond, and one query tile 2^22 of them.  The head dimension is 8
# so that the tensors stay small.  Closed forms: q is orthogonal to every key, so all scores are 0 and P_ij = 1 / (p_i + 1);
# the first half of the keys has k = +1 in column 0 and v = 0, the second k = -1 and v = 1 in every column.
N_LONG, ROWS = 1 << 29, 128


def _room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB of free device memory")


def _long_window():
    D = 8
    k, v = (torch.zeros(1, 1, N_LONG, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[:, :, :, 0] = 1.0
    k[:, :, N_LONG // 2:, 0] = -1.0
    v[:, :, N_LONG // 2:] = 1.0
    q = torch.ones(1, 1, ROWS, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 0.0
    seen = torch.arange(N_LONG - ROWS, N_LONG, dtype=torch.float64, device="cuda") + 1
    x = (seen - N_LONG // 2) / seen  # the weight of the second half
    o = x.to(torch.bfloat16)[None, None, :, None].expand(1, 1, ROWS, D).contiguous()
    lse = torch.log(seen).float().reshape(1, 1, ROWS)
    return q, k, v, o, torch.ones_like(q), lse, seen, x


def _check_long_dq(dq, delta, x, scale):
    # dP = 0 or 8, delta = 8 x, dS = P (dP - delta): dQ_0 = scale (-8 x (1 - x) - 8 (1 - x) x).  x is within 2^-22 of 1/2
    # and o in bf16 is 1/2, P within 2^-11 of 2^-29 (its row's LSE in fp32): dS is +-4 P rounded to bf16, off by 2^-8 + 2^-11
    # of its value and the same for all keys of a half.  A step's 128 equal summands are m 2^-20 with m of 8 bits, sums
    # below 4 hold 2^-22 exactly: each of the 2^21 steps of a half is off by 2^-23 of a share of 2^-20 if m is not 1, by
    # nothing if it is (4 P is 2^-27 up to 2^-19 of its value, and the nearest bf16 value is 2^-27 itself).  Below 2^-6.
    want = -16 * x * (1 - x) * scale
    assert torch.isfinite(dq).all() and not dq[..., 1:].any()
    assert ((dq[0, 0, :, 0].double() - want).abs() <= 2.0 ** -6 * want.abs()).all()
    assert ((delta[0, 0].double() - 8 * x).abs() <= 2.0 ** -7 * 8 * x).all()


@pytest.mark.gpu
def test_a_query_tile_of_the_longest_window():
    """dQ of one query tile: its store waits for all of the tile's steps."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    _room(40)
    q, k, v, o, dO, lse, _, x = _long_window()
    dq = torch.full(q.shape, float("nan"), device="cuda")
    dq, delta = fa.fa_window_backward_dq(q, k, v, o, dO, lse, N_LONG, scale=0.5, dq=dq)
    assert fa.fa_device_status() == 0
    _check_long_dq(dq, delta, x, 0.5)
