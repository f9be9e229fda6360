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
