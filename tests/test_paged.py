"""A paged cache (append with rotation, decode, gather; bf16 and 4-bit pages) against the definition in 64 bits, through the
library's Python entry points; refusals through the C ABI."""
import ctypes
import math

import pytest
import torch

from attention_tiled_fwd_gb300 import _native as nat
from helpers import cuda_or_skip
from paged_ref import (FOUR, append_reference, decode_reference, once, page_values, place, put, quantised, rows_of, turned,
                       unit_values)
from window_ref import check, check_lse, window_reference


# ------------------------------------------------------------------ no GPU: the reference, the layout, refusals
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("of_values", [False, True])
def test_a_unit_holds_every_code_and_scale_once(D, of_values):
    byte, shift, scale = place(D, of_values)
    assert sorted((2 * byte + shift // 4).flatten().tolist()) == list(range(16 * D))
    assert sorted(scale[:, ::32].flatten().tolist()) == list(range(D // 2))
    for p in range(16):  # a byte belongs to one position, so rows can enter one by one
        others = torch.cat((byte[:p], byte[p + 1:])).flatten().tolist()
        assert not set(byte[p].tolist()) & set(others)


def test_places_by_hand():
    # D = 64: two groups, two words a lane.  Key position 9, channel 45: half 1, group 1, lane 4 * 1 + 13 // 8 = 5,
    # word (1 * 32 + 5) * 2 + 1 = 75, nibble 5 -> byte 302, shift 4; scale 9 * 2 + 1
    byte, shift, scale = place(64, False)
    assert (int(byte[9, 45]), int(shift[9, 45]), int(scale[9, 45])) == (302, 4, 19)
    # value: lane 4 * (13 // 4) + 1 // 2 = 12, word (32 + 12) * 2 + 1 = 89, odd position: nibble 4 + 1 -> byte 358, shift 4;
    # scale (4 * 2 + 1) * 2 + 1
    byte, shift, scale = place(64, True)
    assert (int(byte[9, 45]), int(shift[9, 45]), int(scale[9, 45])) == (358, 4, 19)


def test_once_rounds_once():
    one = 1.0 + 2.0 ** -8  # halfway between the bf16 values 1 and 1 + 2^-7
    y = torch.tensor([one, one + 2.0 ** -40, one - 2.0 ** -40, -one - 2.0 ** -40, 0.3, -5.1e-3], dtype=torch.float64)
    assert once(y)[:4].tolist() == [1.0, 1.0 + 2.0 ** -7, 1.0, -1.0 - 2.0 ** -7]
    assert torch.equal(once(y)[4:], y[4:].float().bfloat16())


def test_quantised_rows_by_hand():
    y = torch.zeros(1, 32)
    y[0, :5] = torch.tensor([-7.0, 3.5, 0.5, 1.5, -2.4])
    codes, scale = quantised(y.bfloat16())
    assert float(scale) == 1.0 and codes[0, :6].tolist() == [1, 12, 8, 10, 6, 8]  # 3.5, 0.5 and 1.5 go to even
    assert quantised(torch.zeros(1, 32).bfloat16())[1].item() == 0
    y[0, 9] = math.inf
    assert math.isnan(quantised(y.bfloat16())[1].item())


def test_put_and_read_back_in_four_bits():
    g = torch.Generator().manual_seed(1)
    for of_values in (False, True):
        pages = torch.randint(0, 256, (3, 2, 32, 9 * 4), generator=g, dtype=torch.uint8)
        before = unit_values(pages, 64, of_values)[0]
        table = torch.tensor([[2, 0]])
        row = torch.randn(2, 64, generator=g).bfloat16()
        put(pages, table, 0, 37, row, of_values)
        after, s = unit_values(pages, 64, of_values)
        codes, scales = quantised(row)
        assert torch.equal(after[0, :, 5], (codes.double() - 8) * scales.double().repeat_interleave(32, -1))
        assert float((after[0, :, 5] - row.double()).abs().max()) <= 0.5 * float(s[0, :, 5].max()) * (1 + 2.0 ** -8)
        others = torch.ones(3, 2, 32, dtype=torch.bool)
        others[0, :, 5] = False
        assert torch.equal(after.nan_to_num()[others], before.nan_to_num()[others])


def test_rotation_keeps_lengths_and_angles():
    from attention_tiled_fwd_gb300 import rotation_table
    cos, sin = rotation_table(50, 8, base=100.0, device="cpu")
    assert cos.dtype == torch.float32 and cos.shape == (50, 4)
    assert torch.allclose(cos[7, 2], torch.tensor(math.cos(7 * 100.0 ** -0.5))) and torch.equal(sin[0], torch.zeros(4))
    x = torch.randn(3, 5, 16, generator=torch.Generator().manual_seed(2)).double()
    for inter in (False, True):
        # scores depend on the distance of two positions alone
        a = turned(x[:1], torch.tensor([5, 6, 7, 8, 9]), cos, sin, 8, inter), turned(x[1:2], torch.tensor([1, 2, 3, 4, 5]), cos, sin, 8, inter)
        b = turned(x[:1], torch.tensor([45, 46, 47, 48, 49]), cos, sin, 8, inter), turned(x[1:2], torch.tensor([41, 42, 43, 44, 45]), cos, sin, 8, inter)
        assert torch.allclose((a[0] * a[1]).sum(-1), (b[0] * b[1]).sum(-1), atol=1e-5)
        assert torch.equal(a[0][..., 8:], x[:1, :, 8:])


@pytest.fixture(scope="module")
def lib():
    from attention_tiled_fwd_gb300 import build
    build.build()
    return nat.load()


A = 4096  # a fake, 16-byte aligned address: the call must be refused before it is touched
SIZES = dict(B=2, Hq=4, Hkv=2, n=3, D=64, rot=64, interleaved=0, positions=128, n_pages=9, page=32, slots=4, rows=128,
             window=128, sinks=0, scale=0.1, dtype=nat.FA_BF16, ptr=A, table=A, lens=A, q=A, q_out=A, cos=A, counts=None,
             strides=None)


def _append(lib, **kw):
    a = dict(SIZES, **kw)
    return lib.fa_paged_append(a["q"], a["ptr"], A, a["strides"], a["cos"], a["cos"], a["table"], a["lens"], a["counts"],
                               a["q_out"], A, A, *(a[n] for n in ("B", "Hq", "Hkv", "n", "D", "rot", "interleaved", "positions",
                                                                 "n_pages", "page", "slots", "dtype")), None)


def _decode(lib, **kw):
    a = dict(SIZES, **kw)
    return lib.fa_paged_decode(a["ptr"], A, A, a["table"], a["lens"], A, A,
                               *(a[n] for n in ("B", "Hq", "Hkv", "n", "D", "n_pages", "page", "slots", "window", "sinks",
                                                "scale", "dtype")), A, 1 << 30, None)


def _gather(lib, **kw):
    a = dict(SIZES, **kw)
    return lib.fa_paged_gather(a["ptr"], A, a["table"], a["lens"], A, A,
                               *(a[n] for n in ("B", "Hkv", "rows", "D", "n_pages", "page", "slots", "dtype")), None)


@pytest.mark.parametrize("call", [_append, _decode, _gather])
def test_refusals_of_every_call(lib, call):
    for kw, code in ((dict(B=0), "SHAPE"), (dict(B=65536), "SHAPE"), (dict(Hkv=0), "SHAPE"), (dict(n_pages=0), "SHAPE"),
                     (dict(slots=0), "SHAPE"), (dict(page=8), "SHAPE"), (dict(page=48), "SHAPE"), (dict(page=512), "SHAPE"),
                     (dict(page=256, slots=(1 << 15) + 1, positions=1 << 30), "SHAPE"), (dict(n_pages=(1 << 30)), "SHAPE"),
                     (dict(D=96), "HEAD_DIM"), (dict(D=192), "HEAD_DIM"), (dict(D=0), "SHAPE"), (dict(dtype=nat.FA_F32), "DTYPE"),
                     (dict(dtype=3), "DTYPE"), (dict(ptr=None), "NULL"), (dict(ptr=A + 8), "ALIGN"), (dict(table=None), "NULL")):
        assert call(lib, **kw) == getattr(nat, "FA_ERR_" + code), kw


def test_refusals_of_one_call(lib):
    def refused(call, code, **kw):
        assert call(lib, **kw) == getattr(nat, "FA_ERR_" + code), kw

    refused(_append, "SHAPE", n=0)
    refused(_append, "SHAPE", q=None)              # heads of a q that is not given
    refused(_append, "SHAPE", Hq=0)
    refused(_append, "SHAPE", rot=24)
    refused(_append, "SHAPE", rot=80)
    refused(_append, "SHAPE", rot=-16)
    refused(_append, "SHAPE", positions=127)       # fewer angles than positions
    refused(_append, "SHAPE", B=65535, n=1 << 15)
    refused(_append, "NULL", cos=None)
    refused(_append, "NULL", q_out=None)
    refused(_append, "ALIGN", cos=A + 4)
    refused(_append, "ALIGN", strides=(ctypes.c_longlong * 9)(0, 0, 64, 0, 0, 64, 0, 0, 68))
    refused(_append, "DEVICE_PTR", rot=0, cos=None)  # nothing is left but that the pointers are fakes
    for call in (_decode, _append):
        refused(call, "NULL" if call is _append else "DEVICE_PTR", lens=None)
    refused(_decode, "SHAPE", n=0)
    refused(_decode, "SHAPE", n=17)
    refused(_decode, "SHAPE", Hq=3)
    refused(_decode, "SHAPE", window=0)
    refused(_decode, "SHAPE", sinks=-1)
    refused(_decode, "SCALE", scale=0.0)
    refused(_decode, "SCALE", scale=math.nan)
    refused(_gather, "SHAPE", rows=0)
    refused(_gather, "SHAPE", rows=1 << 30)
    out = ctypes.c_size_t(0)
    assert lib.fa_paged_decode_workspace_bytes(2, 4, 2, 1, 64, 32, 4, nat.FA_BF16, None) == nat.FA_ERR_NULL
    assert lib.fa_paged_decode_workspace_bytes(2, 4, 2, 1, 64, 31, 4, nat.FA_BF16, ctypes.byref(out)) == nat.FA_ERR_SHAPE
    assert lib.fa_status_string(nat.FA_ERR_PAGE) != b"unknown status"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [nat.FA_BF16, nat.FA_INT4])
def test_workspace_stays_below_its_bound(lib, D, dtype):
    out = ctypes.c_size_t(0)
    for B, Hq, Hkv, n_q, page, slots in ((1, 1, 1, 1, 16, 1), (1, 32, 8, 16, 256, 1 << 15), (65535, 8, 1, 16, 16, 1000),
                                         (64, 32, 8, 1, 64, 512), (7, 64, 1, 5, 128, 77)):
        assert lib.fa_paged_decode_workspace_bytes(B, Hq, Hkv, n_q, D, page, slots, dtype, ctypes.byref(out)) == nat.FA_OK
        assert out.value <= 16 << 20


def test_pages_of_the_wrong_kind():
    from attention_tiled_fwd_gb300 import _pages, paged_cache
    k, v = paged_cache(3, 2, 16, 64, nat.FA_INT4, device="cpu")
    assert k.shape == (3, 2, 16, 36) and k.dtype == torch.uint8 and not v.any()
    assert paged_cache(3, 2, 16, 64, device="cpu")[0].shape == (3, 2, 16, 64)
    with pytest.raises(ValueError):
        paged_cache(3, 2, 16, 64, nat.FA_F32, device="cpu")
    table = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        _pages(k.to(torch.int32), v, table, None, 1, 0)
    with pytest.raises(ValueError):
        _pages(k[..., :35], v, table, None, 1, 0)
    with pytest.raises(ValueError):
        _pages(k, v, table, None, 1, 0)  # not on the device


# ------------------------------------------------------------------ GPU
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(lens, page, slots, n_pages, seed=0):
    """Pages drawn from all of the pool, -1 where a sequence needs none."""
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    rows = []
    for n in lens:
        need = -(-max(n, 0) // page)
        rows.append([order.pop() for _ in range(need)] + [-1] * (slots - need))
    return _ints(rows)


def _pool(g, n_pages, H, page, D, four):
    """Pages that hold something everywhere."""
    if not four:
        return tuple(_randn(g, n_pages, H, page, D) for _ in range(2))
    out = []
    for _ in range(2):
        units = torch.randint(0, 256, (n_pages, H, page // 16, 9 * D), generator=g, device="cuda", dtype=torch.uint8)
        codes = units[..., :8 * D]
        codes[(codes & 15) == 0] += 1
        codes[(codes >> 4) == 0] += 16
        scales = torch.rand(n_pages, H, page // 16, D // 2, generator=g, device="cuda") * 0.3 + 0.05
        units[..., 8 * D:] = scales.half().view(torch.uint8)
        out.append(units.view(n_pages, H, page, 9 * D // 16))
    return tuple(out)


def _same(a, b):
    """Equal bits (a NaN is one NaN)."""
    if a.dtype == torch.bfloat16:
        return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
    return torch.equal(a, b)


# B, Hq, Hkv, n, page, lens (cycled), D, rot, interleaved
APPENDS = [
    (1, 1, 1, 1, 16, (1,), 64, 64, False), (3, 4, 2, 1, 16, (17, 1, 160), 128, 128, False),
    (2, 6, 3, 5, 32, (5, 77), 64, 32, True), (4, 8, 1, 33, 64, (33, 20, 0, 90), 128, 64, False),
    (2, 3, 3, 40, 16, (49, 40), 256, 256, False), (2, 2, 2, 17, 128, (200, 130), 256, 16, True),
    (5, 16, 4, 3, 256, (2, 3, 4, 300, -1), 128, 128, True), (1, 9, 3, 100, 16, (111,), 64, 0, False),
    (1, 0, 2, 70, 32, (130,), 128, 128, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("case", APPENDS)
def test_append(case, four):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, n, page, lens, D, rot, inter = case
    g = _gen(B + n + D + rot)
    lens = [lens[b % len(lens)] for b in range(B)]
    slots = -(-max(max(lens), 1) // page) + 1
    table = _tables(lens, page, slots, B * slots + 2)
    pages = _pool(g, B * slots + 2, Hkv, page, D, four)
    qkv = _randn(g, B, n, Hq + 2 * Hkv, D).transpose(1, 2)  # one projection's output, token by token
    q, k, v = (qkv[:, :Hq] if Hq else None), qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cos, sin = fa.rotation_table(slots * page, rot) if rot else (None, None)
    want = append_reference(q, k, v, pages, table, lens, cos, sin, rot, inter)
    got = fa.fa_paged_append(k, v, *pages, table, _ints(lens), q=q, cos=cos, sin=sin, interleaved=inter)
    assert fa.fa_device_status() == 0
    assert (got is None) == (q is None)
    for a, b, name in zip((got, *pages), want, ("q", "k_pages", "v_pages")):
        assert a is None or _same(a, b), f"{name}: {int((a != b).sum())} of {a.numel()} differ"


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_append_of_a_padded_batch(four):
    """Sequences with fewer new rows than the tensor has: what is not new stays as it was, zeros in q."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(3)
    lens, counts = [40, 40, 7, 64, 12], [9, 0, 20, -3, 1 << 30]
    table = _tables([64] * 5, 16, 4, 20)
    pages = _pool(g, 20, 2, 16, 128, four)
    q, k, v = _randn(g, 5, 4, 9, 128), _randn(g, 5, 2, 9, 128), _randn(g, 5, 2, 9, 128)
    cos, sin = fa.rotation_table(64, 128)
    want = append_reference(q, k, v, pages, table, lens, cos, sin, 128, False, counts)
    got = fa.fa_paged_append(k, v, *pages, table, _ints(lens), q=q, cos=cos, sin=sin, counts=_ints(counts))
    for a, b in zip((got, *pages), want):
        assert _same(a, b)
    assert not got[1].any() and not got[2, :, :2].any() and got[2, :, 2:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_sums_that_lie_between_two_bf16_values_are_rounded_once(inter):
    """Cosines that put a cos + b sin a hair beside the halfway point of two bf16 values, and far cancellation."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(5)
    n, D = 256, 64
    cos, sin = (torch.randn(n, D // 2, generator=g, device="cuda") for _ in range(2))
    k = _randn(g, 1, 1, n, D)
    i = torch.arange(D // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + D // 2)
    mid = (once(k[0, 0, :, a].double()).float() * (1 + 2.0 ** -8)).double()  # near a halfway point of bf16
    sin[:128] = ((k[0, 0, :128, a].double() * cos[:128].double() - mid[:128]) / k[0, 0, :128, b].double()).float()
    sin[128:] = (k[0, 0, 128:, a].double() * cos[128:].double() / k[0, 0, 128:, b].double()).float()  # sums near 0
    y = turned(k, torch.arange(n, device="cuda"), cos, sin, D, inter)
    assert int((y.float().bfloat16() != once(y)).sum()) > 0 or int((y[..., :128, a].abs() > 0).sum()) > 0
    pages = _pool(g, 16, 1, 16, D, False)
    table = _ints([list(range(16))])
    want = append_reference(None, k, k, pages, table, [n], cos, sin, D, inter)
    fa.fa_paged_append(k, k, *pages, table, _ints([n]), cos=cos, sin=sin, interleaved=inter)
    assert _same(pages[0], want[1])


@pytest.mark.gpu
def test_four_bit_rows_of_all_sizes():
    """Groups of zeros, of tiny and huge values, with an infinity or a NaN."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(7)
    k, v = _randn(g, 1, 2, 48, 64), _randn(g, 1, 2, 48, 64)
    size = torch.tensor([0.0, 1e-9, 3e-7, 1e-5, 1.0, 1e4, 4e5, 1e8, 1e38], device="cuda")
    for t in (k, v):
        t.mul_(size[torch.randint(0, 9, (1, 2, 48, 2), generator=g, device="cuda")].repeat_interleave(32, -1))
        t[0, 0, 5, 7], t[0, 1, 9, 40], t[0, 1, 20, 3] = math.inf, math.nan, -math.inf
    pages = _pool(g, 4, 2, 16, 64, True)
    table = _ints([[3, 1, 2, 0]])
    want = append_reference(None, k, v, pages, table, [48], None, None, 0, False)
    fa.fa_paged_append(k, v, *pages, table, _ints([48]))
    for i, (a, b) in enumerate(zip(pages, want[1:])):
        (x, s), (y, r) = (unit_values(t, 64, i == 1) for t in (a, b))
        assert torch.equal(s.nan_to_num(), r.nan_to_num()) and torch.equal(s.isnan(), r.isnan())
        assert torch.equal(x.nan_to_num(), y.nan_to_num())
    assert int(unit_values(pages[0], 64, False)[1].isnan().sum()) == 3 * 32


@pytest.mark.gpu
def test_four_bit_rows_of_every_magnitude():
    """A group for every finite magnitude of bf16 as its largest one: scales and codes are the definition's, bit by bit."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(8)
    most = torch.arange(0x7f80, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16).float()
    rows = most.repeat_interleave(32) * (2 * torch.rand(32 * len(most), generator=g, device="cuda") - 1)
    rows = rows.view(-1, 32)
    at, sign = (torch.randint(0, m, (len(most),), generator=g, device="cuda") for m in (32, 2))
    rows[torch.arange(len(most), device="cuda"), at] = most * (1 - 2 * sign)
    n = len(most) // 32  # in rows of 8 groups, 4 heads
    k = rows.to(torch.bfloat16).view(1, 4, n, 256)
    v = k.flip(2).contiguous()
    pages, table = _pool(g, 4, 4, 256, 256, True), _ints([[2, 0, 3, 1]])
    want = append_reference(None, k, v, pages, table, [n], None, None, 0, False)
    fa.fa_paged_append(k, v, *pages, table, _ints([n]))
    for a, b in zip(pages, want[1:]):
        assert torch.equal(a, b)
    assert fa.fa_device_status() == 0


# B, Hq, Hkv, n_q, page, lens (cycled), D, window, sinks; window 0: none
DECODES = [
    (1, 1, 1, 1, 16, (1,), 64, 0, 0), (2, 4, 4, 1, 16, (70, 3), 128, 0, 0), (3, 8, 2, 1, 32, (500, 33, 64), 128, 0, 0),
    (4, 8, 1, 1, 64, (1000, 64, 0, 129), 64, 0, 0), (2, 6, 2, 3, 16, (2, 333), 64, 0, 0), (2, 16, 2, 2, 128, (700, 257), 256, 0, 0),
    (3, 8, 2, 5, 256, (900, 4, 256), 128, 0, 0), (1, 32, 1, 1, 64, (2000,), 128, 0, 0), (2, 8, 1, 16, 16, (400, 15), 128, 0, 0),
    (2, 24, 2, 2, 32, (300, 100), 256, 0, 0), (3, 4, 2, 1, 16, (900, 20, 300), 128, 100, 0), (2, 4, 1, 4, 64, (1500, 200), 64, 333, 5),
    (2, 8, 2, 3, 256, (2500, 2), 128, 130, 4), (2, 6, 3, 2, 32, (1200, 40), 256, 64, 130), (2, 2, 2, 1, 16, (3000, 600), 64, 1, 1),
    (40, 8, 4, 1, 16, (5, 300, 90, 0, 1000), 64, 0, 0), (9, 16, 2, 1, 64, (3000, 17, 800), 128, 0, 0), (1, 4, 4, 1, 64, (4096,), 256, 0, 0),
    (1, 4, 2, 2, 16, (9000,), 64, 5000, 40), (2, 8, 2, 3, 64, (9000, 300), 128, 5000, 5), (1, 2, 1, 1, 32, (7000,), 256, 4500, 70),
    (40, 16, 8, 1, 16, (900, 20, 300), 64, 100, 3),
    # clusters of four and of two
    (20, 8, 4, 1, 16, (300, 90, 0, 200), 64, 0, 0), (60, 4, 2, 1, 32, (500, 1, 130), 128, 0, 0), (8, 8, 8, 2, 16, (150, 40), 256, 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("room", [20, 8500])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("case", DECODES)
def test_decode(case, four, room):
    """`room`: positions behind the longest sequence; lists of few tiles are shared by the CTAs of a cluster, others cut."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, n_q, page, lens, D, window, sinks = case
    g = _gen(sum(case[:5]) + D)
    lens = [lens[b % len(lens)] for b in range(B)]
    slots = -(-(max(lens) + room) // page)
    n_pages = sum(-(-n // page) for n in lens) + 2
    table = _tables(lens, page, slots, n_pages)
    pages = _pool(g, n_pages, Hkv, page, D, four)
    q = _randn(g, B, Hq, n_q, D)
    w = window or slots * page
    ref = decode_reference(q, pages, table, lens, w, sinks, 0.11)
    # what no row sees: behind the sequences' ends, and between the sinks and the window
    keep = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for j in range(n):
            if j < sinks or j > n - n_q - w:
                keep[int(table[b, j // page]), j % page] = True
        if window:
            for s in range(slots):
                if not keep[int(table[b, s]), :].any():
                    table[b, s] = -1
    for i, t in enumerate(pages):
        if not four:
            t.masked_fill_(~keep[:, None, :, None], math.nan)
            continue
        scales = t.view(n_pages, Hkv, page // 16, 9 * D)[..., 8 * D:].view(torch.float16)
        at = place(D, i == 1)[2][:, ::32].to("cuda")  # [16, D / 32]
        for p in range(page):
            scales[:, :, p // 16][..., at[p % 16]] = torch.where(keep[:, p, None, None], scales[:, :, p // 16][..., at[p % 16]], math.nan)
    o, lse = fa.fa_paged_decode(q, *pages, table, _ints(lens), window=window or None, sinks=sinks, scale=0.11)
    assert fa.fa_device_status() == 0
    check(o, ref["o"], ref["o_bound"], "O")
    check_lse(lse, ref["lse"], "LSE")
    again = fa.fa_paged_decode(q, *pages, table, _ints(lens), window=window or None, sinks=sinks, scale=0.11)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_gather(D, four):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    for page, rows, lens in ((16, 100, [37, 0, 100, 1]), (64, 130, [130, 500, 64, -4]), (256, 7, [300, 3])):
        g = _gen(D + page)
        slots = -(-max(max(lens), rows) // page)
        n_pages = len(lens) * slots
        table = _tables([slots * page] * len(lens), page, slots, n_pages)
        pages = _pool(g, n_pages, 3, page, D, four)
        k, v = (torch.full((len(lens), 3, rows, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        got = fa.fa_paged_gather(*pages, table, _ints(lens), k=k, v=v)
        assert got[0] is k and got[1] is v and fa.fa_device_status() == 0
        for i, t in enumerate((k, v)):
            values = page_values(pages[i], D, i == 1)
            for b, n in enumerate(lens):
                n = max(0, min(n, rows))
                assert torch.equal(t[b, :, :n], rows_of(values, table, b, n).float().bfloat16())  # products of 15 bits: fp32 holds them
                assert bool((t[b, :, n:] == 7).all())
        whole = fa.fa_paged_gather(*pages, table)
        assert whole[0].shape[2] == slots * page
        assert torch.equal(whole[0], torch.stack([rows_of(page_values(pages[0], D, False), table, b, slots * page).float().bfloat16()
                                                  for b in range(len(lens))]))


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_pages_that_the_pool_has_not(four):
    """Entries outside the pool where rows are needed: zeros are read, nothing is written, and the status word says so."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(21)
    pages = _pool(g, 6, 2, 16, 128, four)
    table = _ints([[0, 1, 2], [3, 6, 5], [4, -7, 1 << 30]])
    lens = [40, 41, 48]
    q = _randn(g, 3, 4, 1, 128)
    ref = decode_reference(q, pages, table, lens, 48, 0, 0.1)
    o, lse = fa.fa_paged_decode(q, *pages, table, _ints(lens), scale=0.1)
    assert fa.fa_device_status() == nat.FA_ERR_PAGE and fa.fa_device_status() == 0
    check(o, ref["o"], ref["o_bound"], "O")
    check_lse(lse, ref["lse"], "LSE")
    k, _ = fa.fa_paged_gather(*pages, table, _ints(lens))
    assert fa.fa_device_status() == nat.FA_ERR_PAGE
    assert not k[1, :, 16:32].any() and not k[2, :, 16:48].any() and k[1, :, 32:41].any()
    new = _randn(g, 3, 2, 30, 128)
    want = append_reference(None, new, new, pages, table, lens, None, None, 0, False)
    fa.fa_paged_append(new, new, *pages, table, _ints(lens))
    assert fa.fa_device_status() == nat.FA_ERR_PAGE
    for a, b in zip(pages, want[1:]):
        assert _same(a, b)
    # rows past the table's last page
    want = append_reference(None, new[:1], new[:1], pages, table[:1], [60], None, None, 0, False)
    fa.fa_paged_append(new[:1], new[:1], *pages, table[:1].contiguous(), _ints([60]))
    assert fa.fa_device_status() == nat.FA_ERR_PAGE
    for a, b in zip(pages, want[1:]):
        assert _same(a, b)
    for far in ((1 << 31) - 1, -(1 << 31)):
        fa.fa_paged_append(new[:1], new[:1], *pages, table[:1].contiguous(), _ints([far]))
        assert fa.fa_device_status() == (nat.FA_ERR_PAGE if far > 0 else 0)
    for a, b in zip(pages, want[1:]):
        assert _same(a, b)


@pytest.mark.gpu
def test_decode_lengths_are_clamped():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(23)
    pages = _pool(g, 12, 2, 16, 64, False)
    table = _ints(torch.arange(12).view(3, 4).tolist())
    q = _randn(g, 3, 2, 1, 64)
    a, b = (fa.fa_paged_decode(q, *pages, table, _ints(x)) for x in ([-5, 65, 1 << 30], [0, 64, 64]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert not a[0][0].any() and torch.isinf(a[1][0]).all()
    c = fa.fa_paged_decode(q, *pages, table)
    assert torch.equal(c[0][1:], b[0][1:]) and fa.fa_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("crowd", [0, 600])
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_shows_where_it_is_seen_and_nowhere_else(D, four, crowd):
    """`crowd`: further sequences, so many that lists are cut into runs instead of being shared by clusters."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(25)
    pages = _pool(g, 40, 1, 16, D, four)
    table = _ints([list(range(20))] + [list(range(20, 40))] * (1 + crowd))
    q = _randn(g, 2 + crowd, 2, 4, D)
    lens = _ints([300] * (2 + crowd))
    base = fa.fa_paged_decode(q, *pages, table, lens, window=50, sinks=3)
    for which in (0, 1):
        for j in (1, 3, 200, 246, 247, 249, 250, 298, 299):
            bad = [t.clone() for t in pages]
            page, p = j // 16, j % 16
            if four:
                at = place(D, which == 1)[2][p, 0]
                bad[which].view(40, 1, 1, 9 * D)[page, 0, 0, 8 * D:].view(torch.float16)[at] = math.nan
            else:
                bad[which][page, 0, p, 5] = math.nan
            o, lse = fa.fa_paged_decode(q, *bad, table, lens, window=50, sinks=3)
            for i in range(4):
                seen = j <= 296 + i and (j < 3 or j > 246 + i)
                assert bool(o[0, :, i].isnan().any()) == seen, (which, j, i)
                if not seen:
                    assert torch.equal(o[0, :, i], base[0][0, :, i]) and torch.equal(lse[0, :, i], base[1][0, :, i])
            assert torch.equal(o[1:], base[0][1:])


@pytest.mark.gpu
@pytest.mark.parametrize("scale_v", [1e-6, 1e-3, 30.0, 3e4])
def test_four_bit_values_of_any_size(scale_v):
    """Scales from fp16's subnormals to its largest values: the weights' products with them stay in range."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(27)
    pages = list(_pool(g, 40, 2, 16, 128, True))
    scales = pages[1].view(40, 2, 1, 9 * 128)[..., 8 * 128:].view(torch.float16)
    scales.copy_((scales.float() * scale_v * torch.exp2(torch.randint(-3, 2, scales.shape, generator=g, device="cuda"))).half())
    table, lens = _ints([list(range(40))]), [633]
    q = _randn(g, 1, 8, 1, 128)
    ref = decode_reference(q, pages, table, lens, 640, 0, 0.2)
    o, lse = fa.fa_paged_decode(q, *pages, table, _ints(lens), scale=0.2)
    # the products P s in fp16 may be subnormal: 2^-24 of a step against the largest scale's 2^0 at least
    check(o, ref["o"], ref["o_bound"] + 2.0 ** -11 * float(scales.float().max()), "O")
    check_lse(lse, ref["lse"], "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("q_size", [1e-4, 300.0, 3e37])
def test_four_bit_queries_of_any_size(q_size):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(29)
    pages = _pool(g, 10, 1, 16, 64, True)
    table, lens = _ints([list(range(10))]), [155]
    q = (torch.randn(1, 4, 2, 64, generator=g, device="cuda") * q_size).bfloat16()
    q[0, 0, 0] = 0
    ref = decode_reference(q, pages, table, lens, 160, 0, 0.1 / q_size)
    o, lse = fa.fa_paged_decode(q, *pages, table, _ints(lens), scale=0.1 / q_size)
    check(o, ref["o"], ref["o_bound"], "O")
    check_lse(lse, ref["lse"], "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_a_prompt_in_chunks_then_tokens(four):
    """A server's life of two sequences: chunks of a prompt enter the pages, their attention runs on the rows read back,
    then tokens are decoded one and three at a time against the pages; every row against attention over what the pages hold."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(31)
    B, Hq, Hkv, N, D, W, S, page = 2, 8, 2, 400, 128, 96, 4, 32
    slots = -(-N // page)
    kind = fa.FA_INT4 if four else fa.FA_BF16
    pages = fa.paged_cache(B * slots, Hkv, page, D, kind)
    table = _tables([N] * B, page, slots, B * slots)
    cos, sin = fa.rotation_table(slots * page, D)
    qkv = _randn(g, B, N, Hq + 2 * Hkv, D).transpose(1, 2)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    turned_q = once(turned(q, torch.arange(N, device="cuda"), cos, sin, D, False))

    def enter(r0, r1):
        return fa.fa_paged_append(k[:, :, r0:r1], v[:, :, r0:r1], *pages, table, _ints([r1] * B), q=q[:, :, r0:r1], cos=cos, sin=sin)

    for r0, r1 in ((0, 150), (150, 390)):
        qr = enter(r0, r1)
        assert torch.equal(qr, turned_q[:, :, r0:r1])
        K, V = fa.fa_paged_gather(*pages, table, _ints([r1] * B), rows=r1)
        o, lse = fa.fa_window_forward(qr, K, V, W, S)
        ref = window_reference(qr, K, V, W, S, 1 / math.sqrt(D))
        check(o, ref["o"], ref["o_bound"], f"O {r0}..{r1}")
    for r0, r1 in ((390, 391), (391, 394), (394, 400)):
        qr = enter(r0, r1)
        o, lse = fa.fa_paged_decode(qr, *pages, table, _ints([r1] * B), window=W, sinks=S)
        ref = decode_reference(qr, pages, table, [r1] * B, W, S, 1 / math.sqrt(D))
        check(o, ref["o"], ref["o_bound"], f"O {r0}..{r1}")
        check_lse(lse, ref["lse"], f"LSE {r0}..{r1}")
    if not four:  # and the pages hold the rotated rows themselves
        K, V = fa.fa_paged_gather(*pages, table, _ints([N] * B), rows=N)
        assert torch.equal(K, once(turned(k, torch.arange(N, device="cuda"), cos, sin, D, False))) and torch.equal(V, v)
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_captured_steps_follow_their_lengths(four):
    """A captured decoding step (append, decode, gather), replayed as the sequences grow."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(33)
    table = _tables([640] * 3, 64, 10, 30)
    mine, other = (_pool(_gen(34), 30, 2, 64, 128, four) for _ in range(2))
    q, k, v = _randn(g, 3, 8, 1, 128), _randn(g, 3, 2, 1, 128), _randn(g, 3, 2, 1, 128)
    cos, sin = fa.rotation_table(640, 128)
    lens = _ints([1, 1, 1])
    rows = torch.zeros(2, 3, 2, 640, 128, dtype=torch.bfloat16, device="cuda")

    def step(pages):
        qr = fa.fa_paged_append(k, v, *pages, table, lens, q=q, cos=cos, sin=sin)
        return (qr, *fa.fa_paged_decode(qr, *pages, table, lens), *fa.fa_paged_gather(*pages, table, lens, k=rows[0], v=rows[1]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(mine)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(mine)
    step(other)
    for now in ([0, 5, 17], [1, 6, 18], [640, 321, 64], [2, 639, 65]):
        for t in (q, k, v):
            t.copy_(_randn(g, *t.shape))
        lens.copy_(_ints(now))
        graph.replay()
        got = [t.clone() for t in captured]
        for a, b in zip(got, step(other)):
            assert _same(a, b)
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
def test_two_streams_and_a_stream_that_is_not_the_current_one():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(35)
    pages = _pool(g, 200, 2, 64, 128, False), _pool(g, 200, 2, 64, 128, True)
    table, lens = _tables([3000, 3000, 3000], 64, 48, 200), _ints([3000, 2900, 5])
    q = _randn(g, 3, 8, 2, 128)
    want = [fa.fa_paged_decode(q, *p, table, lens) for p in pages]
    streams = [torch.cuda.Stream() for _ in pages]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[fa.fa_paged_decode(q, *p, table, lens, stream=s) for _ in range(5)] for p, s in zip(pages, streams)]
    torch.cuda.synchronize()
    for results, w in zip(got, want):
        for o, lse in results:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.gpu
def test_two_host_threads():
    """Two threads, each with its stream and its sequences, step at the same time: what one of them alone does."""
    import threading
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    cos, sin = fa.rotation_table(4096, 128)

    def start(seed):
        g = _gen(seed)
        pages = _pool(g, 130, 2, 64, 128, seed % 2 == 1)
        table = _tables([4096, 4096], 64, 64, 130)
        return pages, table, _ints([100, 4000 - seed]), [_randn(g, 2, h, 1, 128) for h in (8, 2, 2)]

    def steps(state, out):
        pages, table, lens, (q, k, v) = state
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(40):
                qr = fa.fa_paged_append(k, v, *pages, table, lens, q=q, cos=cos, sin=sin)
                out.append((qr, *fa.fa_paged_decode(qr, *pages, table, lens)))
                lens += 1
            torch.cuda.current_stream().synchronize()

    alone, together = [[], []], [[], []]
    states = [start(i) for i in (0, 1, 0, 1)]
    torch.cuda.synchronize()
    for i in range(2):
        steps(states[2 + i], alone[i])
    threads = [threading.Thread(target=steps, args=(states[i], together[i])) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(alone, together):
        assert len(a) == len(b) == 40
        for x, y in zip(a, b):
            assert all(torch.equal(m, n) for m, n in zip(x, y))
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_pools_beyond_32_bit_offsets(four):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    D, page, H = 256, 256, 8
    row = 9 * D // 16 if four else 2 * D
    n_pages = (5 << 30) // (H * page * row)
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB")
    g = _gen(37)
    shape, kind = ((n_pages, H, page, row), torch.uint8) if four else ((n_pages, H, page, D), torch.bfloat16)
    pages = [torch.zeros(shape, dtype=kind, device="cuda") for _ in range(2)]
    at = [n_pages - 1, 0, n_pages - 2]
    table = _ints([at])
    k, v, q = _randn(g, 1, H, 600, D), _randn(g, 1, H, 600, D), _randn(g, 1, 2 * H, 1, D)
    fa.fa_paged_append(k, v, *pages, table, _ints([600]))
    small = [t[at].clone() for t in pages]
    few = _ints([[0, 1, 2]])
    want = append_reference(None, k, v, [torch.zeros_like(t) for t in small], few, [600], None, None, 0, False)
    for a, b in zip(small, want[1:]):
        assert torch.equal(a, b)
    a, b = fa.fa_paged_decode(q, *pages, table, _ints([600])), fa.fa_paged_decode(q, *small, few, _ints([600]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = fa.fa_paged_gather(*pages, table, _ints([600])), fa.fa_paged_gather(*small, few, _ints([600]))
    assert torch.equal(a[0][:, :, :600], b[0][:, :, :600]) and torch.equal(a[1][:, :, :600], b[1][:, :, :600])
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
def test_rows_of_other_strides():
    """Broadcast heads, every other row, a batch of one with an odd batch stride; and shared pages that are only read."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(39)
    table = _tables([64, 64], 16, 4, 8)
    base = _randn(g, 2, 1, 40, 128)
    k, v = base.expand(2, 3, 40, 128)[:, :, ::2], _randn(g, 2, 20, 3, 128).transpose(1, 2)
    odd = _randn(g, 5, 3, 20, 128)[2:3].as_strided((1, 3, 20, 128), (13, 20 * 128, 128, 1), 2 * 3 * 20 * 128)
    for kk, vv, t in ((k, v, table), (odd, v[:1], table[:1].contiguous())):
        pages = _pool(g, 8, 3, 16, 128, False)
        lens = [33, 20][:kk.shape[0]]
        want = append_reference(None, kk, vv, pages, t, lens, None, None, 0, False)
        fa.fa_paged_append(kk, vv, *pages, t, _ints(lens))
        assert _same(pages[0], want[1]) and _same(pages[1], want[2])
    shared = _ints([[0, 1, 2], [0, 1, 3]])
    q = _randn(g, 2, 6, 1, 128)
    ref = decode_reference(q, pages, shared, [40, 48], 64, 0, 0.1)
    check(fa.fa_paged_decode(q, *pages, shared, _ints([40, 48]), scale=0.1)[0], ref["o"], ref["o_bound"], "shared pages")


@pytest.mark.gpu
def test_binding_refusals():
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(41)
    pages, table, lens = _pool(g, 4, 2, 16, 64, False), _ints([[0, 1, 2, 3]]), _ints([50])
    q, k = _randn(g, 1, 4, 3, 64), _randn(g, 1, 2, 3, 64)
    cos, sin = fa.rotation_table(64, 64)
    fa.fa_paged_append(k, k, *pages, table, lens, q=q, cos=cos, sin=sin)
    for bad in (dict(q=q, q_out=q), dict(cos=cos), dict(q_out=q), dict(q=q, cos=cos, sin=sin[:, :16].contiguous()),
                dict(counts=_ints([1, 2]))):
        with pytest.raises(ValueError):
            fa.fa_paged_append(k, k, *pages, table, lens, **bad)
    with pytest.raises(fa.FAError) as e:
        fa.fa_paged_append(k, k, *pages, table, lens, cos=cos[:63].contiguous(), sin=sin[:63].contiguous())
    assert e.value.code == nat.FA_ERR_SHAPE
    with pytest.raises(fa.FAError) as e:
        fa.fa_paged_append(_randn(g, 1, 2, 3, 68)[..., :64], k, *pages, table, lens)
    assert e.value.code == nat.FA_ERR_ALIGN
    with pytest.raises(ValueError):
        fa.fa_paged_append(k.transpose(2, 3).contiguous().transpose(2, 3), k, *pages, table, lens)
    with pytest.raises(ValueError):
        fa.fa_paged_append(k, k, *pages, table, None)
    with pytest.raises(TypeError):
        fa.fa_paged_append(k.half(), k, *pages, table, lens)
    with pytest.raises(TypeError):
        fa.fa_paged_decode(q, *pages, table, lens.long())
    with pytest.raises(ValueError):
        fa.fa_paged_decode(_randn(g, 1, 3, 3, 64), *pages, table, lens)
    with pytest.raises(ValueError):
        fa.fa_paged_decode(q, pages[0], pages[1][:3], table, lens)
    with pytest.raises(ValueError):
        fa.fa_paged_decode(q, *pages, table.expand(2, -1), lens)
    long = _ints([list(range(4)) * 50])
    with pytest.raises(fa.FAError) as e:
        fa.fa_paged_decode(q, *pages, long, lens, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == nat.FA_ERR_WORKSPACE
    with pytest.raises(ValueError):
        fa.fa_paged_gather(*pages, table, lens, k=k)
    with pytest.raises(fa.FAError) as e:
        fa.fa_paged_gather(*pages, table, lens, rows=0)
    assert e.value.code == nat.FA_ERR_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("case", [(700, 2, 1, 1, 16, 64, lambda b: b % 40), (5000, 1, 1, 1, 16, 64, lambda b: 17 * b % 50),
                                  (3, 4, 4, 1, 64, 64, lambda b: 90000 - 40000 * b)])
def test_decode_of_many_and_of_long_sequences(case, four):
    """More sequences than a CTA has threads, lengths of zero among them; and lists that go over many CTAs."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    B, Hq, Hkv, n_q, page, D, length = case
    lens = [length(b) for b in range(B)]
    g = _gen(B)
    slots = -(-max(lens) // page)
    n_pages = sum(-(-n // page) for n in lens) + 1
    table, pages = _tables(lens, page, slots, n_pages), _pool(g, n_pages, Hkv, page, D, four)
    q = _randn(g, B, Hq, n_q, D)
    ref = decode_reference(q, pages, table, lens, slots * page, 0, 0.2)
    o, lse = fa.fa_paged_decode(q, *pages, table, _ints(lens), scale=0.2)
    assert fa.fa_device_status() == 0
    check(o, ref["o"], ref["o_bound"], "O")
    check_lse(lse, ref["lse"], "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,n", [(1, 1300000), (16, 82000)])
def test_four_bit_runs_over_the_whole_grid(Hkv, n):
    """So many tiles that all CTAs have runs of many: one list over all of them, and several lists."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    g = _gen(43)
    page, D = 256, 64
    slots = -(-n // page)
    pages = _pool(g, slots, Hkv, page, D, True)
    table = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)[None]
    q = _randn(g, 1, 2 * Hkv, 1, D)
    k, v = (page_values(p, D, i == 1) for i, p in enumerate(pages))
    s = unit_values(pages[1], D, True)[1]
    o, lse = fa.fa_paged_decode(q, *pages, table, _ints([n]), scale=0.3)
    assert fa.fa_device_status() == 0
    for h in range(Hkv):  # head by head: 64 bits of all of them at once are much memory
        kb, vb, sb = (rows_of(t[:, h:h + 1], table, 0, n)[0] for t in (k, v, s))
        score = 0.3 * q[0, 2 * h:2 * h + 2, 0].double() @ kb.T
        L = torch.logsumexp(score, -1)
        P = torch.exp(score - L[:, None])
        O, A = P @ vb, P @ vb.abs()
        # as in paged_ref: a warp adds up less than 4096 keys here, the rest are 608 partials (2^-24 of A each)
        bound = (2.0 ** -10 + 2.0 ** -11) * A + 2.0 ** -8 * O.abs() + 2.0 ** -11 * (P @ sb)
        check(o[0, 2 * h:2 * h + 2, 0], O, bound, f"O of head {h}")
        check_lse(lse[0, 2 * h:2 * h + 2, 0], L, f"LSE of head {h}")
