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
