"""The paged-cache operators as they are measured.

A cache of keys and values lies in pages of `page` positions; a table names each sequence's pages, and `lens` says
how many keys each sequence holds.  Pages hold bf16 (``bits`` 16) or 4-bit values (``bits`` 4).  Three operators:

* ``append``  the n newest rows of each sequence (views of one projection's output, token by token): their q and k
              are rotated by their positions, k and v go to their pages.  4-bit pages are read back by ``gather`` in
              the same pass, as a prompt's attention does, so that the outputs are the values that the cache holds.
* ``decode``  attention of the n_q <= 16 newest rows of each sequence against its pages, grouped heads.
* ``gather``  the keys and values of each sequence, from its pages into contiguous bf16 rows.

Row i of n rows sits at position p = len - n + i; rows before position 0 do not exist (their outputs are zeros, their
log-sum-exp -inf).  Row p sees key j iff j <= p and (j < sinks or j > p - window); window 0 stands for no window.

4-bit pages: units of 16 positions, each 8 D bytes of codes and then D bytes of scales.  A value is
scale * (code - 8), one fp16 scale for 32 channels of one position; the order inside a unit is in `_unpacked`.
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ cases
def _case(name, op, bits, B, Hq, Hkv, n, page, min_len, max_len, D, window=0, sinks=0, rot=0, interleaved=False):
    return {"name": name, "op": op, "bits": bits, "B": B, "Hq": Hq, "Hkv": Hkv, "n": n, "page": page,
            "min_len": min_len, "max_len": max_len, "D": D, "window": window, "sinks": sinks, "rot": rot,
            "interleaved": interleaved}


def listed():
    return [
        # one decoding step of a serving batch: latency
        _case("append_tokens", "append", 16, 64, 32, 8, 1, 16, 1, 1024, 128, rot=128),
        # four prompts at the length of the default benchmark
        _case("append_prompts", "append", 16, 4, 16, 4, 4096, 64, 4096, 4096, 128, rot=128),
        # one step of a small batch into 4-bit pages, half of each head rotated in neighbouring pairs
        _case("append4_tokens", "append", 4, 16, 16, 4, 1, 16, 1, 200, 64, rot=32, interleaved=True),
        # a chunk of two long prompts behind what they hold already, ragged
        _case("append4_chunk", "append", 4, 2, 32, 8, 2000, 64, 9001, 16384, 128, rot=128),
        # one token of one sequence: latency
        _case("decode_one", "decode", 16, 1, 16, 4, 1, 16, 3001, 3001, 128),
        # a serving batch of ragged sequences
        _case("decode_batch", "decode", 16, 64, 32, 8, 1, 64, 900, 16384, 128),
        # drafted tokens, a window and sinks that are no multiple of a page, three query heads a key head
        _case("decode_odd", "decode", 16, 7, 6, 2, 3, 32, 2, 5000, 64, window=1001, sinks=5),
        # one token of one sequence in 4 bits: latency
        _case("decode4_one", "decode", 4, 1, 16, 4, 1, 16, 3001, 3001, 128),
        # the serving batch in 4 bits, in small pages
        _case("decode4_batch", "decode", 4, 64, 32, 8, 1, 16, 900, 16384, 128),
        # the 32K context of the long workload, many sequences, two rows each
        _case("decode4_long", "decode", 4, 48, 32, 8, 2, 128, 9000, 32768, 128),
        # one short prompt read back
        _case("gather_short", "gather", 16, 1, 16, 4, 1, 16, 777, 777, 128),
        # long prompts read back from 4 bits for their next chunk
        _case("gather4_long", "gather", 4, 4, 32, 8, 1, 64, 20000, 32768, 128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above, no larger than the largest listed one of its operator."""
    op, bits = rng.choice(("append", "decode", "decode", "gather")), rng.choice((16, 4))
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op and c["bits"] == bits)
    while True:
        hkv = rng.choice((1, 2, 3, 4, 8))
        hq = hkv * rng.choice((1, 2, 3, 4, 8))
        d = rng.choice((64, 128, 128, 256))
        b = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 32768)
        lo = rng.choice((hi, rng.randint(0, hi)))
        n, window, sinks, rot = 1, 0, 0, 0
        if op == "append":
            n = rng.choice((1, 3, 4, _log_int(rng, 5, 4096)))
            rot = rng.choice((d, d, d // 2, 16))
            hi = max(hi, n)
        elif op == "decode":
            n = rng.choice((1, 1, 1, 2, 3, 5, 16))
            window = rng.choice((0, 0, _log_int(rng, 32, 8192)))
            sinks = rng.choice((0, 1, 4, 5, 130)) if window else 0
        case = _case(None, op, bits, b, hq, hkv, n, rng.choice((16, 32, 64, 128, 256)), lo, hi, d, window, sinks, rot,
                     rng.random() < 0.3)
        if b * hkv * hi * d > 1.7e9 or b * hq * n * d > 2e8:  # rows laid out in full, as the plain forms have them
            continue
        if work(case)["bytes"] <= most:
            del case["name"]
            return case


def _lens(case, seed):
    """Sequence lengths spread evenly over [min_len, max_len], in an order of the seed."""
    b, lo, hi = case["B"], case["min_len"], case["max_len"]
    lens = [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]
    random.Random(seed).shuffle(lens)
    return lens


def _slots(case):
    """Pages of the longest sequence."""
    return max(1, -(-case["max_len"] // case["page"]))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    B, Hq, Hkv, n, D, bits = (case[k] for k in ("B", "Hq", "Hkv", "n", "D", "bits"))
    held = 2 * D if bits == 16 else D // 2 + D // 16  # bytes of one cached row
    lens = _lens(case, 0)
    if case["op"] == "gather":
        return {"bytes": 2 * Hkv * sum(lens) * (held + 2 * D), "flops": 2 * Hkv * sum(lens) * D if bits == 4 else 0}
    if case["op"] == "append":
        new = sum(min(n, x) for x in lens)
        moved = new * (Hq * 4 * D + 2 * Hkv * (2 * D + held)) + 4 * case["rot"] * new
        flops = 3 * new * (Hq + Hkv) * case["rot"]
        if bits == 4:  # 32 channels' largest, a product, a rounding; and read back
            moved += 2 * Hkv * sum(lens) * (held + 2 * D)
            flops += 6 * new * Hkv * D + 2 * Hkv * sum(lens) * D
        return {"bytes": moved, "flops": flops}
    keys = pairs = 0
    for x in lens:
        w, s = case["window"] or 1 << 40, case["sinks"]
        lo = max(0, x - n - w + 1)
        keys += x - lo + min(lo, s)
        pairs += sum(min(p + 1, w + min(s, max(0, p + 1 - w))) for p in range(max(0, x - n), x))
    return {"bytes": 2 * Hkv * keys * held + B * Hq * n * (4 * D + 4), "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ inputs
def _pool(g, case, n_pages):
    """Pages as a running server has them: every position written by somebody."""
    Hkv, page, D = case["Hkv"], case["page"], case["D"]
    if case["bits"] == 16:
        return torch.randn((n_pages, Hkv, page, D), generator=g, device="cuda", dtype=BF16)
    # normal values at about 0.3 deviations a step, the scales of 32 channels' largest
    units = torch.empty((n_pages, Hkv, page // 16, 9 * D), dtype=torch.uint8, device="cuda")
    steps = torch.randn((*units.shape[:3], 16 * D), generator=g, device="cuda", dtype=torch.float16)
    code = steps.mul_(3.2).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
    units[..., : 8 * D] = code[..., ::2] | (code[..., 1::2] << 4)
    scale = torch.rand((*units.shape[:3], D // 2), generator=g, device="cuda", dtype=F32) * 0.2 + 0.22
    units[..., 8 * D:] = scale.to(torch.float16).view(torch.uint8)
    return units.view(n_pages, Hkv, page, 9 * D // 16)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, Hq, Hkv, n, D, page = (case[k] for k in ("B", "Hq", "Hkv", "n", "D", "page"))
    lens, slots = _lens(case, seed), _slots(case)
    need = [-(-x // page) for x in lens]
    n_pages = sum(need) + 3
    order = list(range(n_pages))
    random.Random(seed + 1).shuffle(order)
    rows, at = [], 0
    for k in need:  # the pages of a sequence lie anywhere in the pool; unused entries are -1
        rows.append(order[at:at + k] + [-1] * (slots - k))
        at += k
    x = {"k_pages": _pool(g, case, n_pages), "v_pages": _pool(g, case, n_pages),
         "table": torch.tensor(rows, dtype=torch.int32, device="cuda"),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if case["op"] == "append":
        # one projection's output [B, n, heads, D], seen head by head
        qkv = torch.randn((B, n, Hq + 2 * Hkv, D), generator=g, device="cuda", dtype=BF16).transpose(1, 2)
        x["q"], x["k"], x["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        r = case["rot"]
        angle = torch.arange(slots * page, device="cuda", dtype=F64)[:, None] * torch.pow(
            10000.0, -torch.arange(0, r, 2, device="cuda", dtype=F64) / r)
        x["cos"], x["sin"] = angle.cos().to(F32), angle.sin().to(F32)
    elif case["op"] == "decode":
        x["q"] = torch.randn((B, Hq, n, D), generator=g, device="cuda", dtype=BF16)
        x["workspace"] = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")  # no call takes more
    if case["op"] == "gather" or (case["op"] == "append" and case["bits"] == 4):
        x["k_rows"], x["v_rows"] = (torch.zeros((B, Hkv, slots * page, D), dtype=BF16, device="cuda") for _ in range(2))
    return x


def prepare(case, seed):
    return {**_inputs(case, seed), "case": case}


# ------------------------------------------------------------------ plain forms
def _ordered(codes, D, of_values):
    """Bytes of codes [..., 8 D] of units as [..., 16, D / 2]: two channels each, the lower one in the low nibble.

    They lie in 32-bit words, w = min(4, D / 32) of them beside each other for w groups of 32 channels:
      keys    [position / 8][group / w][position % 8][channel % 32 / 8][group % w] a word of 8 channels
      values  [position / 8][group / w][channel % 32 / 4][position % 8 / 2][group % w] a word of 4 channels of an even
              position and then of the odd one behind it"""
    lead, w = codes.shape[:-1], min(4, D // 32)
    if of_values:
        codes, order = codes.reshape(*lead, 2, D // 32 // w, 8, 4, w, 2, 2), (0, 3, 5, 1, 4, 2, 6)
    else:
        codes, order = codes.reshape(*lead, 2, D // 32 // w, 8, 4, w, 4), (0, 2, 1, 4, 3, 5)
    return codes.permute(*range(len(lead)), *(len(lead) + i for i in order)).reshape(*lead, 16, D // 2)


def _ordered_scales(scales, D, of_values):
    """Scales [..., D / 2] of units as [..., 16, D / 32]; they lie as [position][group] for keys, as
    [position / 2][group][position % 2] for values."""
    if of_values:
        scales = scales.unflatten(-1, (8, D // 32, 2)).transpose(-1, -2)
    return scales.reshape(*scales.shape[:scales.dim() - (3 if of_values else 1)], 16, D // 32)


def _unpacked(pages, D, of_values):
    """The values of 4-bit pages [..., page, 9 D / 16] as fp32 [..., page, D]."""
    units = pages.reshape(*pages.shape[:-2], -1, 9 * D)
    codes = _ordered(units[..., : 8 * D], D, of_values)
    scales = _ordered_scales(units[..., 8 * D:].view(torch.float16), D, of_values)
    codes = torch.stack((codes & 15, codes >> 4), -1).reshape(*units.shape[:-1], 16, D // 32, 32)
    return ((codes.to(F32) - 8) * scales[..., None].to(F32)).reshape(*pages.shape[:-1], D)


def _once(y):
    """64-bit values rounded to bf16 once: a value whose fp32 lies halfway between two of bf16 is moved to its side."""
    f = y.to(F32)
    side = y - f.to(F64)
    half = (f.view(torch.int32) & 0xFFFF) == 0x8000
    f = torch.where(half & (side != 0), torch.nextafter(f, torch.copysign(torch.full_like(f, math.inf), side.to(F32))), f)
    return f.to(BF16)


def _rotated(state, x, at):
    """x [B, H, n, D] rotated by the angles of positions at [B, n], in 64 bits (bf16 values next to a border)."""
    r = state["case"]["rot"]
    c, s = (state[k][at].to(F64)[:, None] for k in ("cos", "sin"))
    y = x.to(F64)
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if state["case"]["interleaved"] else (y[..., : r // 2], y[..., r // 2:r])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack((a, b), -1).flatten(-2) if state["case"]["interleaved"] else torch.cat((a, b), -1)
    return _once(torch.cat((turned, y[..., r:]), -1))


def _quantised(x):
    """Codes and scales of bf16 rows [..., D]: scale = largest / 7 as fp16, code = x * fp32(1 / scale) rounded to even."""
    y = x.to(F32).unflatten(-1, (-1, 32))
    scale = (y.abs().amax(-1).to(F64) / 7).to(F32).to(torch.float16)
    inverse = torch.where(scale > 0, (1 / scale.to(F64)).to(F32), torch.zeros_like(scale, dtype=F32))
    code = (y.to(F64) * inverse.to(F64)[..., None]).round().clamp(-7, 7) + 8
    return code.flatten(-2), scale


def _append_plain(state):
    c = state["case"]
    B, n, page, D = (c[k] for k in ("B", "n", "page", "D"))
    at = state["lens"].long()[:, None] - n + torch.arange(n, device="cuda")
    there, at = at >= 0, at.clamp(min=0)
    q = _rotated(state, state["q"], at) * there[:, None, :, None]
    k = _rotated(state, state["k"], at)
    b, i = torch.nonzero(there, as_tuple=True)
    p = at[b, i]
    slot, off = state["table"].long()[b, p // page], p % page
    if c["bits"] == 16:
        for new, pages in ((k, state["k_pages"]), (state["v"], state["v_pages"])):
            pages[slot, :, off] = new[b, :, i]
        return q, state["k_pages"], state["v_pages"]
    for new, pages, of_values in ((k, state["k_pages"], False), (state["v"], state["v_pages"], True)):
        code, scale = _quantised(new[b, :, i].transpose(0, 1))
        byte = (code[..., ::2] + 16 * code[..., 1::2]).to(torch.uint8)
        units = pages.view(*pages.shape[:2], page // 16, 9 * D)
        place = _ordered(torch.arange(8 * D, device="cuda"), D, of_values)[off % 16]
        units[slot[:, None], :, off[:, None] // 16, place] = byte.permute(1, 2, 0)
        place = _ordered_scales(torch.arange(D // 2, device="cuda"), D, of_values)[off % 16] + 4 * D
        units.view(torch.float16)[slot[:, None], :, off[:, None] // 16, place] = scale.permute(1, 2, 0)
    return (q, *_gather_plain(state))


def _read(state, name, slots):
    """Pages `slots` [B, s] of each sequence (any entry below 0: some page) as fp32 rows [B, Hkv, s * page, D]."""
    c = state["case"]
    pages = state[name][state["table"].long().gather(1, slots.clamp(min=0)).clamp(min=0)].transpose(1, 2)
    rows = _unpacked(pages, c["D"], name == "v_pages") if c["bits"] == 4 else pages.to(F32)
    return rows.flatten(2, 3)


def _gather_plain(state):
    c = state["case"]
    slots = torch.arange(_slots(c), device="cuda").expand(c["B"], -1)
    held = (state["lens"][:, None] > torch.arange(_slots(c) * c["page"], device="cuda"))[:, None, :, None]
    return tuple(torch.where(held, _read(state, n + "_pages", slots).to(BF16), state[n + "_rows"]) for n in ("k", "v"))


def _decode_plain(state):
    c = state["case"]
    q, lens = state["q"], state["lens"].long()
    B, Hq, n, D = q.shape
    Hkv, page = c["Hkv"], c["page"]
    w, s = c["window"] or 1 << 40, c["sinks"]
    # the pages that any row sees: the sinks', then the window's
    first = (lens - n - w + 1).clamp(min=0) // page
    ahead = min(_slots(c), (w + n - 2) // page + 2)
    slots = first[:, None] + torch.arange(ahead, device="cuda")
    sink = torch.arange(min(-(-s // page), _slots(c)), device="cuda").expand(B, -1)
    slots = torch.cat((torch.where(sink < first[:, None], sink, -1), torch.where(slots < _slots(c), slots, -1)), 1)
    j = (slots[:, :, None] * page + torch.arange(page, device="cuda")).flatten(1)
    pos = lens[:, None] - n + torch.arange(n, device="cuda")
    seen = (j[:, None] >= 0) & (j[:, None] <= pos[:, :, None]) & ((j[:, None] < s) | (j[:, None] > pos[:, :, None] - w))
    k, v = (_read(state, name, slots) for name in ("k_pages", "v_pages"))
    score = torch.matmul(q.to(F32).reshape(B, Hkv, -1, D), k.transpose(2, 3)) / math.sqrt(D)
    score = score.view(B, Hkv, Hq // Hkv, n, -1).masked_fill(~seen[:, None, None], -math.inf).flatten(2, 3)
    m = score.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = (score - m).exp_()
    l = e.sum(-1, keepdim=True)
    o = torch.where(l > 0, torch.matmul(e, v) / l, 0.0)
    return o.view(B, Hq, n, D).to(BF16), (m + l.log()).view(B, Hq, n)


# ------------------------------------------------------------------ the library's calls
def _run_own(state):
    import attention_tiled_fwd_gb300 as fa
    c, pages = state["case"], (state["k_pages"], state["v_pages"], state["table"], state["lens"])
    if c["op"] == "decode":
        return fa.fa_paged_decode(state["q"], *pages, window=c["window"] or None, sinks=c["sinks"],
                                  workspace=state["workspace"])
    if c["op"] == "gather":
        return fa.fa_paged_gather(*pages, k=state["k_rows"], v=state["v_rows"])
    q = fa.fa_paged_append(state["k"], state["v"], *pages, q=state["q"], cos=state["cos"], sin=state["sin"],
                           interleaved=c["interleaved"])
    if c["bits"] == 16:
        return q, state["k_pages"], state["v_pages"]
    return (q, *fa.fa_paged_gather(*pages, k=state["k_rows"], v=state["v_rows"]))


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append_plain, "decode": _decode_plain, "gather": _gather_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_place(D, values):
    """Where a unit holds channel c of position u: (byte, shift) of the code and the index of the scale, [16, D] each."""
    u, c = torch.arange(16)[:, None], torch.arange(D)[None]
    g, w = c // 32, min(4, D // 32)
    eighth = (u // 8 * (D // 32 // w) + g // w) * 32
    if values:
        word = (eighth + 4 * (c % 32 // 4) + u % 8 // 2) * w + g % w
        nibble = 4 * (u % 2) + c % 4
        scale = (u // 2 * (D // 32) + g) * 2 + u % 2
    else:
        word = (eighth + 4 * (u % 8) + c % 32 // 8) * w + g % w
        nibble = c % 8
        scale = u * (D // 32) + g
    return [t.cuda() for t in (4 * word + nibble // 2, 4 * (nibble % 2), scale)]


def _exact_rows(case, x, name, b, n):
    """Rows 0 .. n - 1 of sequence b in 64 bits, [Hkv, n, D]."""
    D, page = case["D"], case["page"]
    used = x["table"][b, : -(-n // page)].long()
    pages = x[name][used].transpose(0, 1)
    if case["bits"] == 16:
        return pages.flatten(1, 2)[:, :n].double()
    unit = pages.reshape(case["Hkv"], -1, 9 * D)
    byte, shift, scale = _exact_place(D, name == "v_pages")
    code = (unit[..., byte] >> shift.to(torch.uint8)) & 15
    s = unit[..., 8 * D:].contiguous().view(torch.float16)[..., scale]
    return ((code.double() - 8) * s.double()).flatten(1, 2)[:, :n]


def _exact_turn(case, x, row, at):
    """One sequence's rows [H, m, D] at positions at [m], rotated pair by pair as complex numbers."""
    r = case["rot"]
    y = row.double().clone()
    first = torch.arange(r // 2, device="cuda") * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else r // 2)
    z = torch.complex(y[..., first], y[..., second]) * torch.complex(x["cos"][at].double(), x["sin"][at].double())
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_4bit(rows):
    """What 4-bit pages hold of rows [H, m, D] in bf16's values (64 bits)."""
    y = rows.double().view(*rows.shape[:-1], -1, 32)
    step = (y.abs().max(-1, keepdim=True).values / 7).to(F32).to(torch.float16).double()
    inverse = torch.where(step > 0, 1 / step, 0.0).to(F32).double()
    return ((y * inverse).round().clamp(-7, 7) * step).view(rows.shape)


def exact(case, seed):
    x = _inputs(case, seed)
    B, Hq, Hkv, n, D, page = (case[k] for k in ("B", "Hq", "Hkv", "n", "D", "page"))
    lens = x["lens"].tolist()
    if case["op"] == "gather":
        out = []
        for name in ("k", "v"):
            t = x[name + "_rows"].double()
            for b, m in enumerate(lens):
                t[b, :, :m] = _exact_rows(case, x, name + "_pages", b, m)
            out.append(t)
        return tuple(out)
    if case["op"] == "append":
        q = torch.zeros((B, Hq, n, D), dtype=F64, device="cuda")
        held = [x[k + ("_pages" if case["bits"] == 16 else "_rows")].double() for k in ("k", "v")]
        for b, m in enumerate(lens):
            new = min(n, m)
            at = torch.arange(m - new, m, device="cuda")
            q[b, :, n - new:] = _exact_turn(case, x, x["q"][b, :, n - new:], at)
            rows = [_exact_turn(case, x, x["k"][b, :, n - new:], at), x["v"][b, :, n - new:].double()]
            for t, r, name in zip(held, rows, ("k_pages", "v_pages")):
                if case["bits"] == 16:
                    t[x["table"][b].long()[at // page], :, at % page] = r.transpose(0, 1)
                else:
                    t[b, :, :m] = _exact_rows(case, x, name, b, m)
                    t[b, :, m - new:m] = _exact_4bit(_once(r))
        return (q, *held)
    o = torch.zeros((B, Hq, n, D), dtype=F64, device="cuda")
    lse = torch.full((B, Hq, n), -math.inf, dtype=F64, device="cuda")
    for b, m in enumerate(lens):
        new = min(n, m)
        if new == 0:
            continue
        K, V = (_exact_rows(case, x, name, b, m) for name in ("k_pages", "v_pages"))
        p, j = torch.arange(m - new, m, device="cuda")[:, None], torch.arange(m, device="cuda")[None]
        seen = (j <= p) & ((j < case["sinks"]) | (p - j < (case["window"] or 1 << 40)))
        q = x["q"][b, :, n - new:].double().view(Hkv, Hq // Hkv, new, D)
        s = torch.einsum("hgnd,hjd->hgnj", q, K) / math.sqrt(D)
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        lse[b, :, n - new:] = torch.logsumexp(s, -1).view(Hq, new)
        o[b, :, n - new:] = torch.einsum("hgnj,hjd->hgnd", torch.softmax(s, -1), V).reshape(Hq, new, D)
    return o, lse
