"""Run one attention shape through the public API a few times, for profilers.

    python -m attention_tiled_fwd_gb300.run_case B H N D [--causal] [--backward]
        [--reps R] [--dtype bf16|f32] [--std S]
    python -m attention_tiled_fwd_gb300.run_case B H N D --window W [--sinks S] [--kv-heads G] [--backward | --tokens]
    python -m attention_tiled_fwd_gb300.run_case B H N D --prefix P [--kv-heads G]
    python -m attention_tiled_fwd_gb300.run_case B H N D --paged PAGE [--four] [--kv-heads G] [--rows n]

Each repetition runs fa_forward and, with --backward, fa_backward_dq and
fa_backward_dkdv, on seeded synthetic inputs (seed 4242, the benchmark's
generator).  With --window it runs fa_window_forward (and fa_window_backward), or
with --tokens fa_window_decode of one new row per sequence against a full cache of
N keys; with --prefix fa_prefix_decode of one new row per sequence behind P shared
keys and N of its own (standard normal inputs, the same seed).  With --paged it
appends N rows to every sequence's pages (with --four 4-bit ones), decodes the last n
(default 1) against them and gathers them.  A profiler pointed at one kernel with a launch skip of 1 sees the
second, warm launch.  Exits non-zero if the device status word reports a
failed wait.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("B", type=int)
    ap.add_argument("H", type=int)
    ap.add_argument("N", type=int)
    ap.add_argument("D", type=int)
    ap.add_argument("--causal", action="store_true")
    ap.add_argument("--backward", action="store_true")
    ap.add_argument("--reps", type=int, default=2)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    ap.add_argument("--std", type=float, default=1.0)
    ap.add_argument("--window", type=int)
    ap.add_argument("--sinks", type=int, default=0)
    ap.add_argument("--kv-heads", type=int)
    ap.add_argument("--tokens", action="store_true")
    ap.add_argument("--prefix", type=int)
    ap.add_argument("--paged", type=int)
    ap.add_argument("--four", action="store_true")
    ap.add_argument("--rows", type=int, default=1)
    a = ap.parse_args(argv)

    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    import attention_tiled_fwd_gb300 as fa
    from synthetic_inputs import make_qkv

    dev = torch.device("cuda:0")
    if a.paged is not None:
        return paged(fa, a, dev)
    if a.window is not None or a.prefix is not None:
        return grouped(fa, a, dev)
    h = make_qkv(a.B, a.H, a.N, a.D, 4242, a.dtype, a.std, with_dO=a.backward)
    q, k, v = (h[n].to(dev) for n in ("q", "k", "v"))
    dO = h["dO"].to(dev) if a.backward else None
    for _ in range(a.reps):
        o, lse = fa.fa_forward(q, k, v, causal=a.causal)
        if a.backward:
            dq, delta = fa.fa_backward_dq(q, k, v, o, dO, lse, causal=a.causal, grad_dtype=torch.bfloat16)
            fa.fa_backward_dkdv(q, k, v, dO, lse, delta, causal=a.causal, grad_dtype=torch.bfloat16)
    return report(fa, a, "causal" if a.causal else "non-causal", "fwd+bwd" if a.backward else "fwd", a.dtype)


def grouped(fa, a, dev) -> int:
    """The windowed and shared-prefix calls, with --kv-heads key heads."""
    G = a.kv_heads or a.H
    g = torch.Generator(device=dev)
    g.manual_seed(4242)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev).bfloat16()

    rows = 1 if a.tokens or a.prefix is not None else a.N
    q, k, v = randn(a.B, a.H, rows, a.D), randn(a.B, G, a.N, a.D), randn(a.B, G, a.N, a.D)
    if a.prefix is not None:
        kp, vp = randn(G, a.prefix, a.D), randn(G, a.prefix, a.D)
    dO = randn(*q.shape) if a.backward else None
    for _ in range(a.reps):
        if a.prefix is not None:
            fa.fa_prefix_decode(q, kp, vp, k, v)
        elif a.tokens:
            fa.fa_window_decode(q, k, v, a.window, a.sinks)
        else:
            o, lse = fa.fa_window_forward(q, k, v, a.window, a.sinks)
            if a.backward:
                fa.fa_window_backward(q, k, v, o, dO, lse, a.window, a.sinks, grad_dtype=torch.bfloat16)
    if a.prefix is not None:
        return report(fa, a, f"kv heads {G}", f"prefix {a.prefix}")
    return report(fa, a, f"kv heads {G}", f"window {a.window} sinks {a.sinks}",
                  "tokens" if a.tokens else "fwd+bwd" if a.backward else "fwd")


def paged(fa, a, dev) -> int:
    """The paged cache's calls, with pages in a random order and rows from one projection's output."""
    G, slots = a.kv_heads or a.H, -(-a.N // a.paged)
    g = torch.Generator(device=dev)
    g.manual_seed(4242)
    pages = fa.paged_cache(a.B * slots, G, a.paged, a.D, fa.FA_INT4 if a.four else fa.FA_BF16, dev)
    table = torch.randperm(a.B * slots, generator=g, device=dev).to(torch.int32).view(a.B, slots)
    lens = torch.full((a.B,), a.N, dtype=torch.int32, device=dev)
    cos, sin = fa.rotation_table(slots * a.paged, a.D, device=dev)
    qkv = torch.randn((a.B, a.N, a.H + 2 * G, a.D), generator=g, device=dev, dtype=torch.bfloat16).transpose(1, 2)
    for _ in range(a.reps):
        q = fa.fa_paged_append(qkv[:, a.H:a.H + G], qkv[:, a.H + G:], *pages, table, lens, q=qkv[:, :a.H], cos=cos, sin=sin)
        fa.fa_paged_decode(q[:, :, -a.rows:].contiguous(), *pages, table, lens, window=a.window, sinks=a.sinks)
        fa.fa_paged_gather(*pages, table, lens)
    return report(fa, a, f"kv heads {G}", f"pages of {a.paged}", "4 bits" if a.four else "bf16")


def report(fa, a, *what) -> int:
    torch.cuda.synchronize()
    st = fa.fa_device_status()
    if st != 0:
        print(f"device status {st}", file=sys.stderr)
        return 1
    print("ok", a.B, a.H, a.N, a.D, *what)
    return 0


if __name__ == "__main__":
    sys.exit(main())
