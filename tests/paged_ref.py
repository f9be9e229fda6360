"""A paged cache in 64 bits, from the definition: rows rotated and put in pages, read back, and attended to; with a bound
on what the library's roundings can do to attention over 4-bit pages.

Over 4-bit pages the weight P and its product with a value's scale are rounded to fp16 (2^-11 each of a product of the sum
A = sum P |v|), codes are exact, and O is stored in bf16.  The kernel adds codes 1 .. 15 and takes 8 sum P off, so its fp32
sums are off against sum P s 8 rather than A: n keys, 16 at a time, n / 16 2^-23 of that, below 2^-11 sum P s up to
n = 4096.  Scores: codes against an fp16 q that holds its bf16 values exactly; below the 2^-13 that bf16 pages have."""
import math

import torch

from window_ref import LSE_TOL, U, attend, bound_o, visible  # noqa: F401

FOUR = torch.uint8


def place(D, of_values):
    """Of position p and channel c of a unit: (byte, shift) of its code, index of its scale; [16, D] each."""
    p, c = torch.arange(16)[:, None].expand(16, D), torch.arange(D)[None].expand(16, D)
    g, w = c // 32, min(4, D // 32)
    if of_values:
        lane, nibble = 4 * (c % 32 // 4) + p % 8 // 2, c % 4 + 4 * (p % 2)
        scale = (p // 2 * (D // 32) + g) * 2 + p % 2
    else:
        lane, nibble = 4 * (p % 8) + c % 32 // 8, c % 8
        scale = p * (D // 32) + g
    word = ((p // 8 * (D // 32 // w) + g // w) * 32 + lane) * w + g % w
    return 4 * word + nibble // 2, 4 * (nibble % 2), scale


def unit_values(pages, D, of_values):
    """Values and scales of 4-bit pages [n, H, page, 9 D / 16] in 64 bits, [n, H, page, D] each."""
    units = pages.reshape(*pages.shape[:2], -1, 9 * D)
    byte, shift, scale = (t.to(pages.device) for t in place(D, of_values))
    code = (units[..., byte].int() >> shift) & 15
    s = units[..., 8 * D:].contiguous().view(torch.float16)[..., scale].double()
    shape = (*pages.shape[:3], D)
    return ((code.double() - 8) * s).reshape(shape), s.reshape(shape)


def page_values(pages, D, of_values):
    return unit_values(pages, D, of_values)[0] if pages.dtype == FOUR else pages.double()


def rows_of(values, table, b, n):
    """The first n rows of sequence b, [H, n, D], from pages' values [n_pages, H, page, D]; pages that the pool has not are
    zeros."""
    page = values.shape[2]
    at = table[b, : -(-n // page)].long()
    there = (at >= 0) & (at < values.shape[0])
    rows = values[at.clamp(0, values.shape[0] - 1)] * there.double()[:, None, None, None]
    rows = torch.where(there[:, None, None, None], rows, torch.zeros_like(rows))
    return rows.transpose(0, 1).flatten(1, 2)[:, :n]


def once(y):
    """64-bit values rounded to bf16 once (to nearest, ties to even): through the next fp32 towards zero with a sticky bit."""
    f = y.float()
    f = torch.where(f.double().abs() > y.abs(), torch.nextafter(f, torch.zeros_like(f)), f)
    sticky = (f.double() != y).int()
    return (f.view(torch.int32) | sticky).view(torch.float32).bfloat16()


def turned(x, pos, cos, sin, rot, interleaved):
    """Rows x [.., n, D] turned by the angles of positions [n]; 64 bits."""
    y = x.double().clone()
    if rot:
        i = torch.arange(rot // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = cos[pos].double(), sin[pos].double()
        ya, yb = y[..., a], y[..., b]
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
    return y


def quantised(y):
    """Codes [.., D] and scales [.., D / 32] (fp16) of bf16 rows."""
    g = y.double().unflatten(-1, (-1, 32))
    most = g.abs().amax(-1)
    s = (most / 7).clamp(max=65504.0).float().half()
    s = torch.where(torch.isfinite(g).all(-1), s, torch.full_like(s, math.nan))
    inv = torch.where(s > 0, (1.0 / s.double()).float().double(), torch.zeros_like(most))
    code = torch.nan_to_num((g * inv[..., None]).round().clamp(-7, 7), nan=0.0)
    return (code + 8).flatten(-2).to(torch.uint8), s


def put(pages, table, b, p, row, of_values):
    """Row [H, D] (bf16) to position p of sequence b, as the pages hold it."""
    page, D = pages.shape[2], row.shape[-1]
    at = int(table[b, p // page])
    if pages.dtype != FOUR:
        pages[at, :, p % page] = row
        return
    unit = pages[at].view(pages.shape[1], -1, 9 * D)[:, p % page // 16]  # [H, 9 D], a view
    codes, scales = quantised(row)
    byte, shift, scale = (t[p % 16].to(pages.device) for t in place(D, of_values))
    for n in (0, 1):  # the channels in the low and in the high nibbles
        own = shift == 4 * n
        keep = unit[:, byte[own]] & (15 << 4 - 4 * n)
        unit[:, byte[own]] = keep | (codes[:, own] << (4 * n))
    unit.view(torch.float16)[:, 4 * D + scale[::32]] = scales


def append_reference(q, k, v, pages, table, lens, cos, sin, rot, interleaved, counts=None):
    """q_out and the pages after fa_paged_append; pages: (k_pages, v_pages), not changed."""
    kp, vp = (t.clone() for t in pages)
    B, Hkv, n, D = k.shape
    q_out = None if q is None else torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
    capacity = table.shape[1] * kp.shape[2]
    for b in range(B):
        m = int(lens[b])
        new = n if counts is None else max(0, min(n, int(counts[b])))
        pos = [(i, m - n + i) for i in range(n - new, n) if 0 <= m - n + i < capacity]
        if not pos:
            continue
        i, p = (torch.tensor(t, device=k.device) for t in zip(*pos))
        if q is not None:
            q_out[b, :, i] = once(turned(q[b, :, i], p, cos, sin, rot, interleaved))
        kk = once(turned(k[b, :, i], p, cos, sin, rot, interleaved))
        for j, (_, at) in enumerate(pos):
            if 0 <= int(table[b, at // kp.shape[2]]) < kp.shape[0]:
                put(kp, table, b, at, kk[:, j], False)
                put(vp, table, b, at, v[b, :, pos[j][0]], True)
    return q_out, kp, vp


def decode_reference(q, pages, table, lens, window, sinks, scale):
    """O, LSE and O's bound of fa_paged_decode."""
    B, Hq, n_q, D = q.shape
    four = pages[0].dtype == FOUR
    G = Hq // pages[0].shape[1]
    k, v = (page_values(p, D, i == 1) for i, p in enumerate(pages))
    s = unit_values(pages[1], D, True)[1] if four else None
    out = {"o": [], "lse": [], "o_bound": []}
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * pages[0].shape[2]))
        pos = torch.arange(n - n_q, n, device=q.device)
        seen = visible(pos, max(n, 1), window, sinks) & (pos[:, None] >= 0)
        any_row = seen.any(0)
        kb, vb = (rows_of(t, table, b, max(n, 1)) for t in (k, v))
        kb, vb = (torch.where(any_row[:, None], t, torch.zeros_like(t)) for t in (kb, vb))  # what is masked may be anything
        O, L, P, A = attend(q[b].double(), kb.repeat_interleave(G, 0), vb.repeat_interleave(G, 0), seen, scale)
        bound = bound_o(O, A)
        if four:
            sb = torch.where(any_row[:, None], rows_of(s, table, b, max(n, 1)), torch.zeros((), dtype=torch.float64, device=q.device))
            bound = (2.0 ** -10 + 2.0 ** -11) * A + U * O.abs() + 2.0 ** -11 * torch.matmul(P, sb.abs().repeat_interleave(G, 0))
        for name, t in (("o", O), ("lse", L), ("o_bound", bound)):
            out[name].append(t)
    return {name: torch.stack(t) for name, t in out.items()}
