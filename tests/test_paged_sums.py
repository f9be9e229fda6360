"""How far the sums of the paged calls may be off: bounds that count roundings and nothing else, where the bounds of
test_paged.py allow for bf16 weights and for accumulators that lose bits with a list's length."""
import math

import pytest
import torch

from helpers import cuda_or_skip
from paged_ref import decode_reference, once, place, rows_of, turned, unit_values
from test_paged import _gen, _ints, _pool, _randn, _tables
from window_ref import U, attend, check, check_lse, visible


def _decode_and_reference(case, g):
    """What fa_paged_decode gives, the reference, and a bound for weights that are right to 2^-15.

    A score adds D products in fp32, each addition off by 2^-24 of sum |q k| scale at most: D 2^-24 S of a weight's own value, and
    as much of their sum.  Weights are held to 2^-15, 2^x to 2^-21, a sum of less than 8192 keys, 16 at a time and then in fp32
    in four warps, to 2^-17: together 2^-14.  O is stored in bf16."""
    import attention_tiled_fwd_gb300 as fa
    B, Hq, Hkv, n_q, page, lens, D, window = case
    lens = [lens[b % len(lens)] for b in range(B)]
    slots = -(-max(lens) // page)
    table = _tables(lens, page, slots, sum(-(-n // page) for n in lens) + 1)
    pages = _pool(g, sum(-(-n // page) for n in lens) + 1, Hkv, page, D, False)
    q, scale = _randn(g, B, Hq, n_q, D), 0.05
    o, lse = fa.fa_paged_decode(q, *pages, table, _ints(lens), window=window, scale=scale)
    G, out = Hq // Hkv, []
    for b, n in enumerate(lens):
        k, v = (rows_of(t.double(), table, b, n).repeat_interleave(G, 0) for t in pages)
        pos = torch.arange(n - n_q, n, device="cuda")
        seen = visible(pos, n, window or n, 0) & (pos[:, None] >= 0)
        O, L, P, A = attend(q[b].double(), k, v, seen, scale)
        S = (torch.matmul(q[b].double().abs(), k.abs().transpose(1, 2)) * scale * seen).amax(-1, keepdim=True)
        out.append((O, L, U * O.abs() + (2 * D * 2.0 ** -24 * S + 2.0 ** -14) * A))
    return (o, lse), [torch.stack(t) for t in zip(*out)]


# B, Hq, Hkv, n_q, page, lens (cycled), D, window: clusters and runs, one row tile and two, masks within a unit
FEW_KEYS = [(1, 4, 1, 1, 16, (5,), 64, None), (2, 2, 2, 1, 16, (3, 64), 128, None), (3, 16, 1, 1, 32, (40, 17, 2), 128, None),
            (2, 2, 1, 3, 16, (77, 50), 64, 30), (2, 8, 1, 2, 64, (128, 70), 256, None), (1, 3, 1, 5, 16, (130,), 256, 40),
            (700, 2, 1, 1, 16, (1, 5, 30, 9), 128, None), (400, 16, 1, 1, 16, (20, 7), 64, None), (1, 1, 1, 1, 256, (6000,), 128, None)]


@pytest.mark.gpu
@pytest.mark.parametrize("case", FEW_KEYS)
def test_bf16_pages_lose_the_output_s_rounding_and_little_else(case):
    cuda_or_skip()
    (o, lse), (O, L, bound) = _decode_and_reference(case, _gen(51 + case[0] + case[6]))
    check(o, O, bound, "O")
    check_lse(lse, L, "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_an_infinite_value_stays_infinite(D):
    """In a row that sees it, with a weight that is a bf16 number (one key, equal scores) or not; other channels as without it."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(53 + D)
    pages = _pool(g, 20, 1, 16, D, False)
    table = _ints([list(range(20))] * 4)
    q = _randn(g, 4, 2, 3, D)
    q[3] = 0  # equal weights
    lens = [1, 40, 300, 300]
    base, _ = fa.fa_paged_decode(q, *pages, table, _ints(lens), scale=0.02)
    for j in (0, 37, 38, 39, 100, 299):
        bad = pages[1].clone()
        bad[j // 16, 0, j % 16, 3], bad[j // 16, 0, j % 16, D - 1] = math.inf, -math.inf
        o, _ = fa.fa_paged_decode(q, pages[0], bad, table, _ints(lens), scale=0.02)
        want = base.clone()
        for b, n in enumerate(lens):
            for i in range(3):
                if j <= n - 3 + i:
                    want[b, :, i, 3], want[b, :, i, D - 1] = math.inf, -math.inf
        assert torch.equal(o, want), j
    assert fa.fa_device_status() == 0


def _one_sequence(q, k_of, v_of, n, scale):
    """O, LSE, sum P |v| and what weighs |q k| most, of rows q [rows, D] over n keys that k_of(i, j), v_of(i, j) give in 64 bits."""
    q, step = q.double(), 1 << 18
    l = torch.zeros(len(q), dtype=torch.float64, device="cuda")
    O, A, S = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(l)
    for i in range(0, n, step):
        k, v = k_of(i, min(n, i + step)), v_of(i, min(n, i + step))
        e = torch.exp(scale * q @ k.T)  # (scores below 50: nothing overflows)
        l, O, A = l + e.sum(-1), O + e @ v, A + e @ v.abs()
        S = torch.maximum(S, (scale * q.abs() @ k.abs().T).amax(-1))
    return O / l[:, None], l.log(), A / l[:, None], S


@pytest.mark.gpu
def test_bf16_sums_over_the_longest_lists():
    """More lists of 2^23 keys than there are CTAs (their sequences share their pages), so most of them are one CTA's: 2^21 keys a
    warp.  Values of one sign, where every bit that an accumulator drops is lost for good.  2^17 additions of tiles to a warp's
    sum, each off by 2^-25 of it: 2^-8 of A; the rest as above."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    g, n, D, page, lists = _gen(57), 1 << 23, 64, 256, 500
    slots = n // page
    k, v = _pool(g, slots, 1, page, D, False)
    v.abs_().add_(1)
    order = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    q = _randn(g, lists, 2, 1, D)
    q[:, 0] = 0  # equal weights
    o, lse = fa.fa_paged_decode(q, k, v, order[None].expand(lists, -1).contiguous(), scale=0.2)
    assert fa.fa_device_status() == 0
    some = [0, 251, lists - 1]
    rows = torch.cat((q[:1, 0, 0], q[some, 1, 0]))
    k, v = (t.view(-1, D) for t in (k, v))  # (the keys' order does not matter)
    O, L, A, S = _one_sequence(rows, lambda i, j: k[i:j].double(), lambda i, j: v[i:j].double(), n, 0.2)
    bound = U * O.abs() + (2 * D * 2.0 ** -24 * S[:, None] + 2.0 ** -8 + 2.0 ** -14) * A
    check(o[:, 0, 0], O[:1].expand(lists, D), bound[:1].expand(lists, D), "O of equal weights")
    check(o[some, 1, 0], O[1:], bound[1:], "O")
    check_lse(lse[some, 1, 0], L[1:], "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_four_bit_sums_over_the_longest_lists(D):
    """As above over 4-bit pages, with values of both signs, so that O is small beside sum P |v|.

    Equal weights are powers of two, so their products with the scales are exact: O is off by the sums alone.  A tensor core's sum of n
    products loses n 2^-26 of itself at most.  The codes' sum is sum P s code, here less than 9 sum P s, as the codes' mean is below 9;
    8 sum P s comes off it every 512 keys of a warp: 9 2^-17 sum P s.  What is left stays for 8192 keys: 2^-13 sum P |v|, which is less
    than 4 sum P s (the mean of |code - 8| is 3.7).  Then it is added up in fp32, 256 times: 2^-16 sum P |v|.  Together less than
    9 2^-14 + 2^-12 of sum P s, whatever the list's length.
    Other weights are rounded twice to 2^-11 as well."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    g, n, page, lists = _gen(59 + D), 1 << 23, 256, {64: 650, 128: 500, 256: 340}[D]
    slots = n // page
    pages = _pool(g, slots, 1, page, D, True)
    order = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
    q = _randn(g, lists, 2, 1, D)
    q[:, 0] = 0  # equal weights
    o, lse = fa.fa_paged_decode(q, *pages, order[None].expand(lists, -1).contiguous(), scale=0.1)
    assert fa.fa_device_status() == 0
    some = [0, lists // 2, lists - 1]
    rows = torch.cat((q[:1, 0, 0], q[some, 1, 0]))

    def values(which):
        return lambda i, j: unit_values(pages[which][i // page:j // page], D, which == 1)[0].view(-1, D)

    O, L, A, S = _one_sequence(rows, values(0), values(1), n, 0.1)
    s = sum(unit_values(pages[1][i:i + 1024], D, True)[1].view(-1, D).sum(0) for i in range(0, slots, 1024)) / n
    bound = U * O.abs() + (9 * 2.0 ** -14 + 2.0 ** -12) * s
    check(o[:, 0, 0], O[:1].expand(lists, D), bound[:1].expand(lists, D), "O of equal weights")
    bound = bound + (2 * D * 2.0 ** -24 * S[:, None] + 2.0 ** -10) * A
    check(o[some, 1, 0], O[1:], bound[1:], "O")
    check_lse(lse[some, 1, 0], L[1:], "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_four_bit_sums_of_values_that_cancel(D):
    """131072 keys a list, most lists one CTA's: O is a few thousandths of sum P |v|, and the codes' sum hundreds of times O.

    Of independent roundings that are off by half a step 2^-11 at most, uniformly, the error's root mean square is 2^-11 / sqrt(3) of a
    product's, and of O's, as the products are independent.  The weights' and the products' are two: 4e-4; 5e-4 with all else.
    O's own rounding is what rounding the reference gives."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g, n, lists = _gen(73 + D), 1 << 17, {64: 650, 128: 500, 256: 340}[D]
    codes = [torch.randint(1, 16, (256, 8 * D * 2), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]  # of 256 units
    pages = []
    for c in codes:
        units = torch.empty((n // 16, 9 * D), dtype=torch.uint8, device="cuda")
        at = torch.randint(0, 256, (2, n // 16), generator=g, device="cuda")
        units[:, :8 * D] = c[at[0]][:, ::2] | c[at[1]][:, 1::2] << 4  # (pairs of any two units' halves: all units differ)
        scales = torch.rand((n // 16, D // 2), generator=g, device="cuda") * 0.2 + 0.22
        units[:, 8 * D:] = scales.half().view(torch.uint8)
        pages.append(units.view(-1, 1, 64, 9 * D // 16))
    q = _randn(g, lists, 1, 1, D)
    o, _ = fa.fa_paged_decode(q, *pages, torch.arange(n // 64, device="cuda", dtype=torch.int32).expand(lists, -1).contiguous())
    assert fa.fa_device_status() == 0
    some = torch.arange(0, lists, 5, device="cuda")
    k, v = (unit_values(t, D, i == 1)[0].view(-1, D) for i, t in enumerate(pages))
    O = _one_sequence(q[some, 0, 0], lambda i, j: k[i:j], lambda i, j: v[i:j], n, 1 / math.sqrt(D))[0]
    size, store, error = (float(t.square().mean().sqrt()) for t in (O, O.float().bfloat16().double() - O, o[some, 0, 0].double() - O))
    assert error < math.hypot(store, 5e-4 * size), (error / size, store / size)


def _four_bit_pages(codes, scales, of_values):
    """Pages [n / 16, 1, 16, 9 D / 16] of rows of one head with these codes [n, D] and scales [n, D / 32]."""
    n, D = codes.shape
    units = torch.zeros((n // 16, 9 * D), dtype=torch.uint8)
    byte, shift, scale = place(D, of_values)
    codes = codes.view(n // 16, 16, D).to(torch.uint8)
    for p in range(16):
        for nibble in (0, 4):
            own = shift[p] == nibble
            units[:, byte[p][own]] |= codes[:, p][:, own] << nibble
        units.view(torch.float16)[:, 4 * D + scale[p, ::32]] = scales.view(n // 16, 16, -1)[:, p].half()
    return units.view(n // 16, 1, 16, 9 * D // 16)


def test_four_bit_pages_of_given_codes():
    g = torch.Generator().manual_seed(61)
    for of_values in (False, True):
        codes, scales = torch.randint(1, 16, (48, 64), generator=g), torch.rand(48, 2, generator=g).half()
        values, s = unit_values(_four_bit_pages(codes, scales, of_values), 64, of_values)
        assert torch.equal(s.view(48, 64), scales.double().repeat_interleave(32, 1))
        assert torch.equal(values.view(48, 64), (codes.double() - 8) * scales.double().repeat_interleave(32, 1))


# the ordinary keys' weight beside the heaviest (log2) and scale, and the scale of the keys of no weight at all
OUTLIERS = [(-12.6, 0.15, 0.1), (-12.6, 0.15, 4096.0), (-14.6, 0.15, 4096.0), (-14.6, 0.15, 16384.0), (-15.3, 0.15, 65504.0),
            (-15.3, 3.2e-4, 0.4), (-12.6, 2e-6, 1.0), (-14.6, 300.0, 1.0), (-14.6, 2.0, 1e-3)]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("weight,size,other", OUTLIERS)
def test_four_bit_scales_of_unlike_size(D, weight, size, other):
    """Thousands of keys of low weight, all alike, so that their roundings do not cancel; before them a few of the largest weight,
    and one for each warp that has no weight and a scale of another size.

    Weights are fp16 times 2^6 beside the heaviest, scales times a power of two 2^up for the largest of a warp's tile (32 keys, 16
    at D = 256), and their products fp16.  So besides 2^-11 of itself a weight is off by 2^-31, a product by 2^-31 2^-up, and a scale by 2^-25
    2^-up; a code is within 7 of 8, and l is 1 at least beside the heaviest.  2^up (2^15 at most) puts the tile's largest scale into
    [2^-4, 2), and where it has to change, as between sizes 32 apart, into [1, 2)."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    n, lists, tile = 4000, 700, 16 if D == 256 else 32
    key = torch.arange(n)
    heavy, none = (key < 4 * tile) & (key % 16 == 0), (key >= 4 * tile) & (key < 8 * tile) & (key % tile == 1)
    ks = torch.where(heavy, 1e-4, torch.where(none, 80.0, -weight * math.log(2.0))) / (0.01 * D)  # a key is -scale in all channels
    kc = torch.full((n, D), 7)
    vc = (torch.arange(D) % 15 + 1).expand(n, D)
    vs = torch.where(none, other, torch.where(heavy, 1e-3 * size, size))
    pages = [_four_bit_pages(c, s[:, None].expand(n, D // 32), i == 1).cuda() for i, (c, s) in enumerate(((kc, ks), (vc, vs)))]
    table = _ints(list(range(n // 16))).expand(lists, -1).contiguous()
    q = torch.ones((lists, 1, 1, D), dtype=torch.bfloat16, device="cuda")
    o, lse = fa.fa_paged_decode(q, *pages, table, _ints([n] * lists), scale=0.01)
    assert fa.fa_device_status() == 0
    k, v = (unit_values(t, D, i == 1)[0].view(n, D) for i, t in enumerate(pages))
    s = unit_values(pages[1], D, True)[1].view(n, D)[:, :1]
    O, L, P, A = attend(q[0, 0].double(), k, v, torch.ones(1, n, dtype=torch.bool, device="cuda"), 0.01)
    step = s.view(-1, tile).amax(1).repeat_interleave(tile)[:, None].clamp(min=2.0 ** -15)  # 2^-up, beside the 16 below
    step[:4 * tile if max(size, other) >= 32 * min(size, other) else n] *= 16
    bound = U * O.abs() + (2.0 ** -10 + 2.0 ** -11) * A + 2.0 ** -11 * (P @ s)
    bound = bound + 7 * (2.0 ** -31 * (s + step).sum() * P.amax() + 2.0 ** -25 * (P @ step))
    check(o[:, 0, 0], O.expand(lists, D), bound.expand(lists, D), "O")
    check_lse(lse[:, 0, 0], L.expand(lists), "LSE")


def test_an_odd_number_of_rotated_channels_is_refused():
    """It would give angles of `rot` for rot / 2 + 1 / 2 pairs, which an append then takes for those of rot + 1."""
    from attention_tiled_fwd_gb300 import rotation_table
    with pytest.raises(ValueError):
        rotation_table(10, 15, device="cpu")


def _near_ties(inter):
    """Rows [1, 1, n, D], cosines and sines whose rotated channels lie 2^-20 to 2^-40 of themselves beside the middle of two bf16 values:
    a cos is the middle itself (a power of two times a number of 9 bits), b sin what it misses."""
    g = torch.Generator().manual_seed(63)
    n, D = 256, 64
    half = (n, D // 2)
    a = 2.0 ** torch.randint(-6, 7, half, generator=g) * (1 - 2.0 * torch.randint(0, 2, half, generator=g))
    middle = 2.0 ** torch.randint(-3, 4, half, generator=g) * (1 + (2 * torch.randint(0, 128, half, generator=g) + 1) / 256)
    b = 2.0 ** torch.randint(-6, 7, half, generator=g)
    sin = middle * a.abs() / b * 2.0 ** torch.randint(-40, -19, half, generator=g) * (1 - 2.0 * torch.randint(0, 2, half, generator=g))
    i = torch.arange(D // 2)
    at = (2 * i, 2 * i + 1) if inter else (i, i + D // 2)
    k = torch.zeros(1, 1, n, D)
    k[0, 0][:, at[0]], k[0, 0][:, at[1]] = a, b
    assert torch.equal(k.bfloat16().float(), k) and torch.equal((a.double() * middle.double()).float().double(), a.double() * middle.double())
    return k.bfloat16(), middle.float(), sin.float(), at


def _turned_once(k, cos, sin, at):
    """Rows [n, D] turned and rounded to bf16 once.  Products of 8 and 24 bits are exact in 64.  Some sums miss the middle by less
    than 2^-53 of it: one that is the middle in 64 bits moves a step to the side of what it dropped (Knuth's TwoSum)."""
    a, b, c, s = k[0, 0][:, at[0]].double(), k[0, 0][:, at[1]].double(), cos.double(), sin.double()
    out = torch.empty(k.shape[2:], dtype=torch.bfloat16, device=k.device)
    for to, x, y in ((at[0], a * c, -b * s), (at[1], b * c, a * s)):
        total = x + y
        part = total - x
        rest = (x - (total - part)) + (y - part)
        middle = (total.float().double() == total) & ((total.float().view(torch.int32) & 0xffff) == 0x8000)
        out[:, to] = once(torch.where(middle & (rest != 0), torch.nextafter(total, rest.sign() * math.inf), total))
    return out


@pytest.mark.parametrize("inter", [False, True])
def test_near_ties_are_near_ties(inter):
    k, cos, sin, at = _near_ties(inter)
    y = turned(k, torch.arange(256), cos, sin, 64, inter)[0, 0][:, at[0]]
    assert torch.equal(_turned_once(k, cos, sin, at)[:, at[0]], once(y))
    # rounded to fp32 first, a good part of those less than 2^-25 beside the middle go the wrong way
    assert int((y.float().bfloat16() != once(y)).sum()) > 1000
    off = (y / (k[0, 0][:, at[0]].double() * cos.double()) - 1).abs()
    assert 2.0 ** -41 < float(off.min()) and float(off.max()) < 2.0 ** -19


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_sums_beside_the_middle_of_two_bf16_values(inter):
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    k, cos, sin, at = (t.cuda() if torch.is_tensor(t) else t for t in _near_ties(inter))
    want = _turned_once(k, cos, sin, at)
    y = turned(k, torch.arange(256, device="cuda"), cos, sin, 64, inter)[0, 0]
    assert int((y.float().bfloat16() != want).sum()) > 1000
    pages, table = _pool(_gen(65), 16, 1, 16, 64, False), _ints([list(range(16))])
    q = fa.fa_paged_append(k, k, *pages, table, _ints([256]), q=k, cos=cos, sin=sin, interleaved=inter)
    assert torch.equal(q[0, 0], want) and torch.equal(pages[0].view(256, 64), want)
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** 127])
def test_a_huge_query_over_keys_of_zeros(four, size):
    """Scores of 0, however large q is: O is the values' mean, and L the logarithm of their number."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(67)
    pages = list(fa.paged_cache(20, 1, 16, 64, fa.FA_INT4 if four else fa.FA_BF16))
    table, lens = _ints([list(range(20))]), _ints([300])
    k, v = torch.zeros(1, 1, 300, 64, dtype=torch.bfloat16, device="cuda"), _randn(g, 1, 1, 300, 64)
    fa.fa_paged_append(k, v, *pages, table, lens)
    if four:  # keys whose codes are 8, of scales that are not 0
        pages[0].view(20, 9 * 64)[:, 8 * 64:] = torch.full((20, 32), 0.5).half().view(torch.uint8).cuda()
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0, 5], q[0, 1, 0, 60] = size, -size
    o, lse = fa.fa_paged_decode(q, *pages, table, lens, scale=1.0)
    values = fa.fa_paged_gather(*pages, table, lens, rows=300)[1][0, 0].double()
    if four:
        values = unit_values(pages[1], 64, True)[0].view(320, 64)[:300]
    O, A = values.mean(0), values.abs().mean(0)
    check(o[0, :, 0], O.expand(2, 64), (U * O.abs() + 2.0 ** -10 * A).expand(2, 64), "O")
    check_lse(lse[0, :, 0], torch.full((2,), math.log(300.0), dtype=torch.float64, device="cuda"), "LSE")
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("size", [1e7, 1e9, 1e14, 1e30])
def test_scores_of_any_size(four, size):
    """Scores so large that one key has all the weight: O is its value, L its score to fp32's precision (D products, 2^-24 of them each)."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(69)
    pages, table, lens = _pool(g, 20, 1, 16, 64, four), _ints([list(range(20))]), [300]
    q = (torch.randn(1, 8, 1, 64, generator=g, device="cuda") * size).bfloat16()
    o, lse = fa.fa_paged_decode(q, *pages, table, _ints(lens), scale=1.0)
    ref = decode_reference(q, pages, table, lens, 320, 0, 1.0)
    check(o, ref["o"], ref["o_bound"], "O")
    assert float((lse.double() / ref["lse"] - 1).abs().max()) < 64 * 2.0 ** -22
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("size", range(22, 31))
def test_large_scores_that_grow_from_tile_to_tile(four, size):
    """Scores about 2^size log2 units, fp32's steps there 2^(size - 23), that grow by 2 to 64 from one 128 keys to the next: O stays among
    the values, L beside the largest score, whichever of the steps a running maximum takes."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g, n, D = _gen(71), 1024, 64
    j = (torch.arange(n) // 128).float()
    q = torch.zeros(1, 6, 1, D, dtype=torch.bfloat16, device="cuda")
    q[0, :, 0, 0] = 2.0 ** size / 28672
    q[0, :, 0, 40] = 2.0 ** torch.arange(1, 7, device="cuda")  # a group of its own
    if four:
        kc, ks = torch.full((n, D), 8), torch.zeros(n, 2)
        kc[:, 0], kc[:, 40], ks[:, 0], ks[:, 1] = 15, 8 + j.long(), 4096.0, 1.0
        pages = [_four_bit_pages(kc, ks, False).cuda()]
        vc, vs = torch.randint(1, 16, (n, D), generator=torch.Generator().manual_seed(1)), torch.full((n, 2), 0.25)
        pages.append(_four_bit_pages(vc, vs, True).cuda())
    else:
        pages = [_randn(g, n // 16, 1, 16, D) for _ in range(2)]
        pages[0].zero_()
        pages[0][..., 0], pages[0].view(n, D)[:, 40] = 28672.0, j.bfloat16().cuda()
    table, lens = _ints([list(range(n // 16))]).expand(700, -1).contiguous(), _ints([n] * 700)
    o, lse = fa.fa_paged_decode(q.expand(700, -1, -1, -1).contiguous(), *pages, table, lens, scale=math.log(2.0))
    v = unit_values(pages[1], D, True)[0].view(n, D) if four else pages[1].view(n, D).double()
    k = unit_values(pages[0], D, False)[0].view(n, D) if four else pages[0].view(n, D).double()
    assert bool(o.isfinite().all()) and bool((o[:, :, 0].double().abs() <= v.abs().amax(0) * (1 + U)).all())
    top = (q[0, :, 0].double() @ k.T).amax(1) * math.log(2.0)
    assert float((lse[:, :, 0].double() / top - 1).abs().max()) < 64 * 2.0 ** -22
    assert fa.fa_device_status() == 0
