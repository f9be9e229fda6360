"""Calls of the paged cache that are refused, or that nothing else makes."""
import pytest
import torch

from attention_tiled_fwd_gb300 import _native as nat
from helpers import cuda_or_skip
from test_paged import _gen, _ints, _pool, _randn


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_append_refuses_outputs_that_share_memory(four):
    """The kernel reads rows while others are written: a row would be rotated twice, or be half of one that is."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(71)
    pages, table, lens = _pool(g, 4, 2, 16, 64, four), _ints([[0, 1, 2, 3]]), _ints([50])
    cos, sin = fa.rotation_table(64, 64)
    rows = _randn(g, 3, 1, 2, 9, 64)  # q, k and what lies behind
    q, k, n = rows[0], rows[1], rows[0].numel()
    flat, before = rows.view(-1), rows.clone()
    held = [t.clone() for t in pages]

    def call(q=q, k=k, pages=pages, **kw):
        return fa.fa_paged_append(k, k, *pages, table, lens, q=q, cos=cos, sin=sin, **kw)

    for at in (8, n // 2, n, n + 64, 2 * n - 8):  # over the end of q, over k
        with pytest.raises(fa.FAError) as e:
            call(q_out=flat[at:at + n].view(1, 2, 9, 64))
        assert e.value.code == nat.FA_ERR_SHAPE
    with pytest.raises(fa.FAError) as e:
        call(pages=(pages[0], pages[0]))
    assert e.value.code == nat.FA_ERR_SHAPE
    torch.cuda.synchronize()
    assert torch.equal(rows, before) and all(torch.equal(a, b) for a, b in zip(pages, held))
    # side by side is well: q_out right behind k, and strided rows that run through one another
    want = call()
    got = call(q_out=flat[2 * n:].view(1, 2, 9, 64))
    assert torch.equal(got, want) and got.data_ptr() == rows[2].data_ptr()
    qkv = rows[:2].permute(1, 3, 0, 2, 4).reshape(1, 9, 4, 64).transpose(1, 2)
    assert torch.equal(call(q=qkv[:, :2], k=qkv[:, 2:]), want)
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
def test_rows_of_one_page_into_another():
    """A sequence that begins as another one's copy: the rows of its last, partly filled page enter a page of its own."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(73)
    pages = _pool(g, 6, 2, 16, 128, False)
    want = [t.clone() for t in pages]
    for t in want:
        t[5, :, :9] = t[1, :, :9]
    k, v = (t[1:2, :, :9] for t in pages)
    fa.fa_paged_append(k, v, *pages, _ints([[0, 5]]), _ints([25]))
    assert all(torch.equal(a, b) for a, b in zip(pages, want)) and fa.fa_device_status() == 0
