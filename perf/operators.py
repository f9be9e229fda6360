"""The windowed and shared-prefix attention operators as they are measured.

Three operators, each a call that a user of the library makes:

* ``window``   attention over a sliding window whose first ``sinks`` keys stay visible.  ``train`` false is a
               prefill: queries are the last Nq of Nk positions, outputs O and LSE.  ``train`` true is a step
               of training: O and the gradients of q, k and v.
* ``token``    the serving form of the same: n_q <= 16 new rows per sequence against a cache of capacity N
               whose sequences hold ``lens`` keys each.
* ``prefix``   n_q <= 16 new rows per sequence of a batch whose sequences share one long prefix and have each
               a cache of their own behind it.

Row i of n query rows sits at position p = len - n + i and sees key j iff j <= p and (j < sinks or
j > p - window); ``prefix`` rows see every prefix key and their own keys j <= p.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
F32 = torch.float32


# ------------------------------------------------------------------ cases
def _window(name, B, Hq, Hkv, Nq, Nk, D, window, sinks, train):
    return {"name": name, "op": "window", "B": B, "Hq": Hq, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "D": D,
            "window": window, "sinks": sinks, "train": train}


def _token(name, B, Hq, Hkv, n_q, N, min_len, max_len, D, window, sinks):
    return {"name": name, "op": "token", "B": B, "Hq": Hq, "Hkv": Hkv, "n_q": n_q, "N": N, "min_len": min_len,
            "max_len": max_len, "D": D, "window": window, "sinks": sinks}


def _prefix(name, B, Hq, Hkv, n_q, P, N, min_len, max_len, D):
    return {"name": name, "op": "prefix", "B": B, "Hq": Hq, "Hkv": Hkv, "n_q": n_q, "P": P, "N": N,
            "min_len": min_len, "max_len": max_len, "D": D}


def listed():
    return [
        # a short prompt: one launch, where latency counts
        _window("prefill_short", 1, 16, 16, 200, 200, 128, 128, 1, False),
        # one chunk of a chunked prefill behind 2048 cached positions, ragged, grouped heads
        _window("prefill_chunk", 4, 16, 4, 500, 2548, 128, 1024, 4, False),
        # the 32K context of the long workload as a prompt, grouped heads, a 4096-key window
        _window("prefill_32k", 1, 32, 8, 32768, 32768, 64, 4096, 4, False),
        # a training step at the shape of the default benchmark, grouped heads
        _window("step_4k", 2, 16, 4, 4096, 4096, 128, 1024, 4, True),
        # the widest head, one key head per query head, no sinks
        _window("step_wide", 1, 8, 8, 8192, 8192, 256, 2048, 0, True),
        # the 32K workload trained with a short window
        _window("step_32k", 1, 32, 32, 32768, 32768, 64, 512, 1, True),
        # nothing a multiple of a tile: odd length, head width, window and sinks, three query heads a key head
        _window("step_odd", 3, 6, 2, 1531, 1531, 80, 300, 5, True),
        # one token of one sequence: latency
        _token("token_one", 1, 16, 4, 1, 4096, 3001, 3001, 128, 1024, 4),
        # a serving batch of ragged sequences, window of 4096 keys
        _token("token_batch", 64, 32, 8, 1, 16384, 900, 16384, 128, 4096, 4),
        # a few sequences behind a short prompt: latency
        _prefix("prefix_small", 5, 16, 4, 1, 777, 128, 1, 100, 128),
        # a serving batch behind one long system prompt
        _prefix("prefix_batch", 64, 32, 8, 1, 16384, 512, 1, 512, 128),
        # many samples of one document, two rows at a time (a drafted token beside the last one)
        _prefix("prefix_large", 256, 32, 8, 2, 32768, 1024, 2, 1024, 128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hkv = rng.choice((1, 2, 3, 4, 8))
    return hkv * rng.choice((1, 2, 3, 4, 8)), hkv


def draw(rng):
    """One more case of the ranges above, no larger than the largest listed one of its operator."""
    op = rng.choice(("window", "window", "train", "train", "token", "prefix"))
    while True:
        hq, hkv = _heads(rng)
        if op in ("window", "train"):
            nk = _log_int(rng, 100, 32768)
            if op == "window":
                nq = nk if rng.random() < 0.5 else _log_int(rng, 17, nk)
            else:
                nq = nk
            case = _window(None, rng.choice((1, 2, 3, 4)), hq, hkv, nq, nk,
                           rng.choice((64, 64, 80, 96, 128, 128, 192, 256)),
                           _log_int(rng, 64, 8192), rng.choice((0, 1, 4, 5, 16, 130)), op == "train")
            cap = 2.5e11 if op == "train" else 1.0e12
        else:
            b, n_q = _log_int(rng, 1, 256), rng.choice((1, 1, 1, 2, 3, 5, 8))
            if op == "token":
                n = _log_int(rng, 64, 32768)
                lo = rng.randint(n_q, n)
                case = _token(None, b, hq, hkv, n_q, n, lo, rng.randint(lo, n), rng.choice((64, 128, 128, 256)),
                              _log_int(rng, 32, 8192), rng.choice((0, 1, 4, 5, 16, 130)))
            else:
                n = _log_int(rng, 16, 2048)
                lo = rng.randint(n_q, n)
                case = _prefix(None, b, hq, hkv, n_q, _log_int(rng, 64, 32768), n, lo, rng.randint(lo, n),
                               rng.choice((64, 128, 128, 256)))
            cap = 2.8e11
            cache = 4 * b * hkv * n * case["D"]
            if cache > 9e9:
                continue
        del case["name"]
        if work(case)["flops"] <= cap:
            return case


def _lens(case, seed):
    """Sequence lengths spread evenly over [min_len, max_len], in an order of the seed."""
    b, lo, hi = case["B"], case["min_len"], case["max_len"]
    lens = [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]
    random.Random(seed).shuffle(lens)
    return lens


# ------------------------------------------------------------------ what a pass cannot do without
def _visible(p, window, sinks):
    """Keys that position p sees."""
    return 0 if p < 0 else min(p + 1, window + min(sinks, max(0, p + 1 - window)))


def work(case):
    B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
    if case["op"] == "window":
        nq, nk = case["Nq"], case["Nk"]
        pairs = B * Hq * sum(_visible(p, case["window"], case["sinks"]) for p in range(nk - nq, nk))
        lo = max(0, nk - nq - case["window"] + 1)
        keys = B * Hkv * (nk - lo + min(lo, case["sinks"]))
        if not case["train"]:
            return {"bytes": 2 * D * (2 * B * Hq * nq + 2 * keys) + 4 * B * Hq * nq, "flops": 4 * D * pairs}
        # q, k, v, dO in; O, dq, dk, dv out; two products forward, five backward
        return {"bytes": 2 * D * (4 * B * Hq * nq + 4 * B * Hkv * nk), "flops": 14 * D * pairs}
    n_q = case["n_q"]
    rows = B * Hq * n_q
    big = case["op"] == "prefix"
    window, sinks = (1 << 40, 0) if big else (case["window"], case["sinks"])
    keys = pairs = 0
    for n in _lens(case, 0):
        lo = max(0, n - n_q - window + 1)
        keys += n - lo + min(lo, sinks)
        pairs += sum(_visible(n - n_q + i, window, sinks) for i in range(n_q))
    keys, pairs = keys * Hkv, pairs * Hq
    if big:
        keys += Hkv * case["P"]
        pairs += rows * case["P"]
    return {"bytes": 2 * D * (2 * rows + 2 * keys) + 4 * rows + 4 * B, "flops": 4 * D * pairs}


# ------------------------------------------------------------------ inputs
def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=BF16)

    B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
    if case["op"] == "window":
        x = {"q": randn(B, Hq, case["Nq"], D), "k": randn(B, Hkv, case["Nk"], D), "v": randn(B, Hkv, case["Nk"], D)}
        if case["train"]:
            x["dO"] = randn(B, Hq, case["Nq"], D)
        return x
    x = {"q": randn(B, Hq, case["n_q"], D), "k": randn(B, Hkv, case["N"], D), "v": randn(B, Hkv, case["N"], D),
         "lens": torch.tensor(_lens(case, seed), dtype=torch.int32, device="cuda")}
    if case["op"] == "prefix":
        x["kp"], x["vp"] = randn(Hkv, case["P"], D), randn(Hkv, case["P"], D)
    return x


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:
        import attention_tiled_fwd_gb300 as fa
        # what a serving loop or a training program keeps between calls: its workspace, its parameters' leaves
        c = case
        if c["op"] == "token":
            n = fa.fa_window_decode_workspace_bytes(c["B"], c["Hq"], c["Hkv"], c["n_q"], c["N"], c["D"], c["window"],
                                                    c["sinks"])
            state["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        elif c["op"] == "prefix":
            n = fa.fa_prefix_decode_workspace_bytes(c["B"], c["Hq"], c["Hkv"], c["n_q"], c["P"], c["N"], c["D"])
            state["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        elif c["train"]:
            for n in ("q", "k", "v"):
                state[n].requires_grad_()
    return state


# ------------------------------------------------------------------ plain forms
def _row_blocks(case):
    """Blocks of query rows with the keys [0, s) and [lo, hi) that any of their rows sees."""
    nq, nk = case["Nq"], case["Nk"]
    for r0 in range(0, nq, 1024):
        r1 = min(nq, r0 + 1024)
        lo = max(0, nk - nq + r0 - case["window"] + 1)
        yield r0, r1, min(lo, case["sinks"]), lo, nk - nq + r1


def _block_probs(case, q, k, r0, r1, s, lo, hi):
    """Scores' softmax of rows [r0, r1) over keys [0, s) and [lo, hi), fp32; q [B, Hkv, G, n, D]."""
    B, Hkv, G, n, D = q.shape
    kk = torch.cat((k[:, :, :s], k[:, :, lo:hi]), 2).to(F32)
    scores = torch.matmul(q.to(F32).reshape(B, Hkv, G * n, D), kk.transpose(2, 3)) / math.sqrt(D)
    p = torch.arange(case["Nk"] - case["Nq"] + r0, case["Nk"] - case["Nq"] + r1, device=q.device)[:, None]
    j = torch.cat((torch.arange(s, device=q.device), torch.arange(lo, hi, device=q.device)))[None, :]
    seen = (j <= p) & ((j < case["sinks"]) | (j > p - case["window"]))
    scores = scores.view(B, Hkv, G, n, -1).masked_fill(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    e = (scores - m).exp_()
    l = e.sum(-1, keepdim=True)
    return e.div_(l).view(B, Hkv, G * n, -1), (m + l.log()).squeeze(-1), kk


def _window_plain(state):
    c = state["case"]
    q, k, v = state["q"], state["k"], state["v"]
    B, Hq, nq, D = q.shape
    Hkv, G = k.shape[1], q.shape[1] // k.shape[1]
    q5 = q.view(B, Hkv, G, nq, D)
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=F32, device=q.device)
    if c["train"]:
        dO5 = state["dO"].view(B, Hkv, G, nq, D)
        dq = torch.empty_like(q)
        dk, dv = torch.zeros_like(k, dtype=F32), torch.zeros_like(v, dtype=F32)
    for r0, r1, s, lo, hi in _row_blocks(c):
        n = r1 - r0
        P, L, kk = _block_probs(c, q5[:, :, :, r0:r1], k, r0, r1, s, lo, hi)
        vv = torch.cat((v[:, :, :s], v[:, :, lo:hi]), 2).to(F32)
        O = torch.matmul(P, vv)
        o.view(B, Hkv, G, nq, D)[:, :, :, r0:r1] = O.view(B, Hkv, G, n, D)
        lse.view(B, Hkv, G, nq)[:, :, :, r0:r1] = L
        if not c["train"]:
            continue
        dO = dO5[:, :, :, r0:r1].to(F32).reshape(B, Hkv, G * n, D)
        gv = torch.matmul(P.transpose(2, 3), dO)
        dS = torch.matmul(dO, vv.transpose(2, 3))
        dS.sub_((dO * O).sum(-1, keepdim=True)).mul_(P).div_(math.sqrt(D))
        dq.view(B, Hkv, G, nq, D)[:, :, :, r0:r1] = torch.matmul(dS, kk).view(B, Hkv, G, n, D)
        gk = torch.matmul(dS.transpose(2, 3), q5[:, :, :, r0:r1].to(F32).reshape(B, Hkv, G * n, D))
        for acc, g in ((dk, gk), (dv, gv)):
            acc[:, :, :s] += g[:, :, :s]
            acc[:, :, lo:hi] += g[:, :, s:]
    return (o, dq, dk.to(BF16), dv.to(BF16)) if c["train"] else (o, lse)


def _joined(parts, D):
    """Softmax-weighted values of several (scores, values) parts of the same rows."""
    m = torch.stack([s.amax(-1) for s, _ in parts]).amax(0)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    l, O = 0, 0
    for s, v in parts:
        e = (s - m[..., None]).exp_()
        l = l + e.sum(-1)
        O = O + torch.matmul(e, v)
    o = torch.where(l[..., None] > 0, O / l[..., None], torch.zeros_like(O))
    return o, m + l.log()


def _token_plain(state):
    c = state["case"]
    q, lens = state["q"], state["lens"].long()
    B, Hq, n_q, D = q.shape
    Hkv = c["Hkv"]
    G, w = Hq // Hkv, min(c["window"], c["N"])
    rows = torch.arange(n_q, device=q.device)
    # the keys that any row sees: the sinks, then those of the window behind them
    j = (lens - n_q - w + 1)[:, None] + torch.arange(w + n_q - 1, device=q.device)
    s = torch.arange(min(c["sinks"], c["N"]), device=q.device).expand(B, -1)
    j = torch.cat((s, torch.where(j < s.shape[1], -1, j)), 1)
    pos = lens[:, None] - n_q + rows
    seen = (j[:, None, :] >= 0) & (j[:, None, :] <= pos[:, :, None]) & (
        (j[:, None, :] < c["sinks"]) | (j[:, None, :] > pos[:, :, None] - c["window"]))
    b = torch.arange(B, device=q.device)[:, None]
    jj = j.clamp(0, c["N"] - 1)
    k = state["k"].transpose(1, 2)[b, jj].transpose(1, 2).to(F32)
    v = state["v"].transpose(1, 2)[b, jj].transpose(1, 2).to(F32)
    scores = torch.matmul(q.to(F32).reshape(B, Hkv, G * n_q, D), k.transpose(2, 3)) / math.sqrt(D)
    scores = scores.view(B, Hkv, G, n_q, -1).masked_fill(~seen[:, None, None], -math.inf).view(B, Hkv, G * n_q, -1)
    o, lse = _joined([(scores, v)], D)
    return o.view(q.shape).to(BF16), lse.view(B, Hq, n_q)


def _prefix_plain(state):
    c = state["case"]
    q, lens = state["q"], state["lens"].long()
    B, Hq, n_q, D = q.shape
    Hkv, N = c["Hkv"], c["N"]
    G = Hq // Hkv
    qf = q.to(F32).reshape(B, Hkv, G * n_q, D)
    # the prefix once for all: the rows of every sequence against it, a key head at a time
    sp = torch.matmul(qf.transpose(0, 1).reshape(Hkv, B * G * n_q, D), state["kp"].to(F32).transpose(1, 2)) / math.sqrt(D)
    mp = sp.amax(-1, keepdim=True)
    ep = sp.sub_(mp).exp_()
    lp = ep.sum(-1, keepdim=True)
    op = torch.matmul(ep, state["vp"].to(F32))

    def by_sequence(t):
        return t.view(Hkv, B, G * n_q, -1).transpose(0, 1)

    mp, lp, op = by_sequence(mp), by_sequence(lp), by_sequence(op)
    j = torch.arange(N, device=q.device)
    pos = lens[:, None] - n_q + torch.arange(n_q, device=q.device)
    seen = j[None, None, :] <= pos[:, :, None]
    ss = torch.matmul(qf, state["k"].to(F32).transpose(2, 3)) / math.sqrt(D)
    ss = ss.view(B, Hkv, G, n_q, N).masked_fill(~seen[:, None, None], -math.inf).view(B, Hkv, G * n_q, N)
    m = torch.maximum(mp, ss.amax(-1, keepdim=True))
    es = ss.sub_(m).exp_()
    w = (mp - m).exp()
    l = es.sum(-1, keepdim=True) + w * lp
    o = (torch.matmul(es, state["v"].to(F32)) + w * op) / l
    return o.reshape(q.shape).to(BF16), (m + l.log()).reshape(B, Hq, n_q)


# ------------------------------------------------------------------ the library's calls
def _run_own(state):
    import attention_tiled_fwd_gb300 as fa
    c = state["case"]
    if c["op"] == "window":
        if not c["train"]:
            return fa.fa_window_forward(state["q"], state["k"], state["v"], c["window"], c["sinks"])
        o = fa.window_attention(state["q"], state["k"], state["v"], c["window"], c["sinks"])
        return (o.detach(),) + torch.autograd.grad(o, (state["q"], state["k"], state["v"]), state["dO"])
    if c["op"] == "token":
        return fa.fa_window_decode(state["q"], state["k"], state["v"], c["window"], c["sinks"], lens=state["lens"],
                                   workspace=state["workspace"])
    return fa.fa_prefix_decode(state["q"], state["kp"], state["vp"], state["k"], state["v"], lens=state["lens"],
                               workspace=state["workspace"])


def run(state):
    if own:
        return _run_own(state)
    return {"window": _window_plain, "token": _token_plain, "prefix": _prefix_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rows(q, keys, values, seen):
    """softmax(q keys^T / sqrt(D)) values and its log-sum-exp over the keys that are seen (64 bits)."""
    s = (q @ keys.mT) / math.sqrt(q.shape[-1])
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, -1)
    return torch.softmax(s, -1) @ values, lse


def _exact_window(case, x):
    nq, nk, W, S = case["Nq"], case["Nk"], case["window"], case["sinks"]
    B, Hq, Hkv, D = (case[n] for n in ("B", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    train = case["train"]
    o = torch.zeros(B, Hq, nq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, Hq, nq, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(o) if train else None
    dk, dv = (torch.zeros(B, Hkv, nk, D, dtype=torch.float64, device="cuda") for _ in range(2)) if train else (None, None)
    for b in range(B):
        for h in range(Hkv):
            K, V = x["k"][b, h].double(), x["v"][b, h].double()
            for r0 in range(0, nq, 2048):
                r1 = min(nq, r0 + 2048)
                p = torch.arange(nk - nq + r0, nk - nq + r1, device="cuda")
                first = max(0, int(p[0]) - W + 1)
                idx = torch.tensor([j for j in range(min(S, first))] + list(range(first, int(p[-1]) + 1)), device="cuda")
                seen = (idx[None] <= p[:, None]) & ((idx[None] < S) | (p[:, None] - idx[None] < W))
                heads = slice(h * G, (h + 1) * G)
                q = x["q"][b, heads, r0:r1].double().requires_grad_(train)
                kk, vv = K[idx].requires_grad_(train), V[idx].requires_grad_(train)
                with torch.set_grad_enabled(train):
                    for g in range(G):
                        out, L = _exact_rows(q[g], kk, vv, seen)
                        o[b, h * G + g, r0:r1] = out.detach()
                        lse[b, h * G + g, r0:r1] = L.detach()
                        if train:
                            gq, gk, gv = torch.autograd.grad(out, (q, kk, vv), x["dO"][b, h * G + g, r0:r1].double())
                            dq[b, h * G + g, r0:r1] = gq[g]
                            dk[b, h].index_add_(0, idx, gk)
                            dv[b, h].index_add_(0, idx, gv)
    return (o, dq, dk, dv) if train else (o, lse)


def _exact_cached(case, x):
    B, Hq, Hkv, D, n_q = (case[n] for n in ("B", "Hq", "Hkv", "D", "n_q"))
    G = Hq // Hkv
    o = torch.zeros(B, Hq, n_q, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, Hq, n_q, dtype=torch.float64, device="cuda")
    prefix = case["op"] == "prefix"
    kp, vp = (x["kp"].double(), x["vp"].double()) if prefix else (None, None)
    for b, n in enumerate(x["lens"].tolist()):
        j = torch.arange(n, device="cuda")
        pos = n - n_q + torch.arange(n_q, device="cuda")
        seen = j[None] <= pos[:, None]
        if not prefix:
            seen &= (j[None] < case["sinks"]) | (pos[:, None] - j[None] < case["window"])
            used = seen.any(0)
            j, seen = j[used], seen[:, used]
        K, V = x["k"][b][:, j].double(), x["v"][b][:, j].double()
        if prefix:
            K, V = torch.cat((kp, K), 1), torch.cat((vp, V), 1)
            seen = torch.cat((torch.ones(n_q, case["P"], dtype=torch.bool, device="cuda"), seen), 1)
        q = x["q"][b].double().view(Hkv, G * n_q, D)
        out, L = _exact_rows(q, K, V, seen.repeat(G, 1)[None])
        o[b], lse[b] = out.view(Hq, n_q, D), L.view(Hq, n_q)
    return o, lse


def exact(case, seed):
    x = _inputs(case, seed)
    with torch.no_grad():
        return _exact_window(case, x) if case["op"] == "window" else _exact_cached(case, x)
