"""How far the sums of paged decode may be off: bounds that count roundings and nothing else, where the bounds of
test_paged.py allow for bf16 weights and for accumulators that lose bits with a list's length."""
import math

import pytest
import torch

from helpers import cuda_or_skip
from paged_ref import rows_of, unit_values
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

    Equal weights are powers of two, so their products with the scales are exact: O is off by the sums alone.  The codes' sum is
    sum P s code, at most 15 sum P s but here, where the codes' mean is below 9, less than 9; the kernel takes 8 sum P s of it every
    4096 keys of a warp, and a tensor core's sum of 4096 products loses 2^-14 of itself at most (n 2^-26): both lose, so their
    difference is off by less than 9 2^-14 sum P s, which does not grow with the list.  512 additions in fp32: 2^-15 sum P |v| < 2^-12 sum P s.
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
