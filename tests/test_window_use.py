"""Windowed attention as programs use it: captured steps, two host threads, recomputed activations."""
import threading

import pytest
import torch

from helpers import cuda_or_skip


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _side(work):
    """Runs work once on another stream, as a warm-up of a capture."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)


@pytest.mark.gpu
@pytest.mark.parametrize("D,N,window,sinks", [(64, 900, 100, 3), (64, 900, 100, 200), (128, 700, 90, 4), (192, 400, 60, 1), (256, 400, 60, 130)])
def test_captured_backward_call_follows_its_inputs(D, N, window, sinks):
    """Both halves of the backward in one call (dK/dV launched as dQ's dependent), replayed with new values."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(D + sinks)
    q, k, v, dO = (_randn(g, 2, h, N, D) for h in (4, 2, 2, 4))

    def work():
        o, lse = fa.fa_window_forward(q, k, v, window, sinks)
        return (o, lse, *fa.fa_window_backward(q, k, v, o, dO, lse, window, sinks))

    _side(work)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = work()
    for _ in range(3):
        for t in (q, k, v, dO):
            t.copy_(_randn(g, *t.shape))
        graph.replay()
        graph.replay()  # the same graph twice in a row: the second starts when the first has ended
        torch.cuda.synchronize()
        for a, b in zip(captured, work()):
            assert torch.equal(a, b)
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_captured_autograd_step_follows_its_inputs(D):
    """window_attention's forward and backward in a graph; no other autograd graph of its leaves is alive."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(D)
    q, k, v = (_randn(g, 2, h, 300, D).requires_grad_() for h in (4, 2, 2))
    dO = _randn(g, 2, 4, 300, D)

    def step(q, k, v):
        o = fa.window_attention(q, k, v, 50, 2)
        return (o.detach(), *torch.autograd.grad(o, (q, k, v), dO))

    _side(lambda: step(q, k, v))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(q, k, v)
    for _ in range(2):
        with torch.no_grad():
            for t in (q, k, v, dO):
                t.copy_(_randn(g, *t.shape))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, step(*(t.detach().clone().requires_grad_() for t in (q, k, v)))):
            assert torch.equal(a, b)
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
def test_two_host_threads():
    """Training steps and decodes from two threads, each on its own stream, give what they give one after the other."""
    import attention_tiled_fwd_gb300 as fa
    cuda_or_skip()
    g = _gen(3)
    sets = []
    for D, window, sinks in ((64, 100, 3), (128, 70, 5)):
        q, k, v = (_randn(g, 2, h, 500, D) for h in (4, 2, 2))
        sets.append((q, k, v, _randn(g, 2, 4, 500, D), _randn(g, 2, 4, 1, D), window, sinks))

    def calls(q, k, v, dO, qt, window, sinks):
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        o = fa.window_attention(*leaves, window, sinks)
        return (o.detach(), *torch.autograd.grad(o, leaves, dO), *fa.fa_window_decode(qt, k, v, window, sinks),
                *fa.fa_prefix_decode(qt, k[0], v[0], k, v))

    expect = [calls(*s) for s in sets]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(2), []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait(30)
                outs = [calls(*sets[i]) for _ in range(20)]
                torch.cuda.current_stream().synchronize()
            for got in outs:
                for a, b in zip(got, expect[i]):
                    assert torch.equal(a, b)
        except BaseException as e:  # noqa: BLE001  (a thread's failure is the test's)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors and not any(t.is_alive() for t in threads), errors
    assert fa.fa_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputed_activations(reentrant):
    """Under torch.utils.checkpoint the forward runs again inside the backward: the same gradients."""
    import attention_tiled_fwd_gb300 as fa
    from torch.utils.checkpoint import checkpoint
    cuda_or_skip()
    g = _gen(4)
    q, k, v = (_randn(g, 1, h, 260, 64).requires_grad_() for h in (4, 2, 2))
    dO = _randn(g, 1, 4, 260, 64)

    def block(q, k, v):
        return fa.window_attention(q * 0.5, k, v, 40, 2)

    want = torch.autograd.grad(block(q, k, v), (q, k, v), dO)
    checkpoint(block, q, k, v, use_reentrant=reentrant).backward(dO)
    for t, w in zip((q, k, v), want):
        assert torch.equal(t.grad, w)
