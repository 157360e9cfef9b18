"""The allocating wrappers of the training operators as calls: what their
results keep alive, other Python threads, a process whose first calls are
captured."""
from __future__ import annotations

import os
import subprocess
import sys
import threading
import time

import pytest
import torch

from tests.test_gpu_parity import fm

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_small_results_keep_little_memory_and_versions_of_their_own():
    """A loss that is kept (for a log) keeps no workspace with it, and the
    results of a call are not views of one another for autograd."""
    m = fm()
    X, W = torch.randn(100, 64, device="cuda").to(BF), torch.randn(5000, 64, device="cuda").to(BF)
    t = torch.randint(0, 5000, (100,), device="cuda")
    loss, lse = m.vocab_loss(X, W, t)
    # 2 x 400 bytes at multiples of 256, and 16 KB of a workspace at most
    assert loss.untyped_storage().nbytes() <= 2 * 512 + (16 << 10)
    assert m.flash_mca_vocab_loss_workspace_bytes(100, 5000, 64) > 16 << 10
    before = lse._version
    loss.mul_(2.0)
    assert lse._version == before and not loss._is_view() and not lse._is_view()
    with torch.inference_mode():
        loss2, lse2 = m.vocab_loss(X, W, t)
    assert torch.equal(loss2 * 2.0, loss) and torch.equal(lse2, lse) and loss2.is_inference()


def test_other_threads_run_while_a_stream_is_full():
    """Calls that wait for room in the stream's queue let other Python threads
    run (the device is kept busy for half a second, ahead of 3000 calls)."""
    m = fm()
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    m.layer_norm(x, w, w)
    torch.cuda.synchronize()
    gaps, stop = [], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.002)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    ticker = threading.Thread(target=tick)
    ticker.start()
    try:
        torch.cuda._sleep(1_000_000_000)
        for _ in range(3000):
            m.layer_norm(x, w, w)
    finally:
        stop.set()
        ticker.join()
    torch.cuda.synchronize()
    assert max(gaps) < 0.25


def test_first_calls_of_a_process_are_captured():
    """The kernels' attributes and residencies are looked up in the first call:
    that call may be one that is being captured."""
    code = """
import torch, flash_mixed_chunk_gb300 as m
torch.manual_seed(0)
g = torch.Generator("cuda").manual_seed(1)
r = lambda *s: (torch.randn(*s, device="cuda", generator=g) / 8).to(torch.bfloat16)
res = {}
for M in (100, 700):
    X, W, Y, Wo, dOut = r(M, 128), r(900, 128), r(M, 256), r(128, 256), r(M, 128)
    Wt, dU, dV, dZ = r(2 * 256 + 64, 128), r(M, 256), r(M, 256), r(M, 64)
    t = torch.randint(0, 900, (M,), device="cuda", generator=g)
    w, dl = torch.ones(128, device="cuda"), torch.rand(M, device="cuda", generator=g)
    def step():
        y, h, mean, rstd = m.layer_norm(X, w, w)
        loss, lse = m.vocab_loss(X, W, t)
        return (y, *m.layer_norm_backward(dOut, h, w, mean, rstd), loss,
                *m.vocab_loss_backward(X, W, t, lse, dl),
                *m.gau_output_backward(Y, Wo, dOut), *m.gau_project_backward(X, Wt, dU, dV, dZ))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0 and "same" in p.stdout, p.stderr[-2000:]


def all_calls(m, r, M):
    """Every operator once, on inputs of the generator r; a list of results."""
    X, W, Y, Wo, dOut = r(M, 128), r(900, 128), r(M, 256), r(128, 256), r(M, 128)
    Wt, dU, dV, dZ = r(2 * 256 + 64, 128), r(M, 256), r(M, 256), r(M, 64)
    t = torch.arange(M, device="cuda") % 900
    w, dl = torch.ones(128, device="cuda"), torch.full((M,), 1.0 / M, device="cuda")

    def step(first):
        y, h, mean, rstd = m.layer_norm(X, w, w)
        loss, lse = m.vocab_loss(X, W, t)
        calls = {"norm": lambda: m.layer_norm(X, w, w)[:1],
                 "norm backward": lambda: m.layer_norm_backward(dOut, h, w, mean, rstd),
                 "loss": lambda: m.vocab_loss(X, W, t),
                 "loss backward": lambda: m.vocab_loss_backward(X, W, t, lse, dl),
                 "output": lambda: m.gau_output_backward(Y, Wo, dOut),
                 "project": lambda: m.gau_project_backward(X, Wt, dU, dV, dZ)}
        return calls[first]

    return X, step


@pytest.mark.parametrize("M", [100, 700])
@pytest.mark.parametrize("first", ["norm", "norm backward", "loss", "loss backward", "output",
                                   "project"])
def test_calls_behind_copies_and_joined_streams(first, M):
    """A call's first kernel behind a copy, a memset and the join of two streams,
    captured and not: what it reads was written there just before."""
    m = fm()
    g = torch.Generator("cuda").manual_seed(3)
    X, step = all_calls(m, lambda *s: (torch.randn(*s, device="cuda", generator=g) / 8).to(BF), M)
    call = step(first)
    keep = X.clone()
    want = [o.clone() for o in call()]
    side = torch.cuda.Stream()

    def joined():
        main = torch.cuda.current_stream()
        X.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            half = keep.float().mul_(0.5)
        X.copy_(keep)                       # a copy, and a kernel on the other stream
        main.wait_stream(side)
        return half, call()

    half, got = joined()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        half, got = joined()
    for _ in range(3):
        X.fill_(7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(half, keep.float() * 0.5)


@pytest.mark.parametrize("explicit", [False, True], ids=["allocating", "into outputs"])
@pytest.mark.parametrize("kind", ["0", "1", "default", "side handle", "side"])
def test_streams_by_handle(kind, explicit):
    """`stream` may be a handle: 0 and 1 are the device's default stream.  The call
    is ordered behind what that stream holds (a delay, then the inputs)."""
    m = fm()
    keep, w = torch.randn(300, 64, device="cuda"), torch.ones(64, device="cuda")
    X, W = torch.randn(300, 64, device="cuda").to(BF), torch.randn(900, 64, device="cuda").to(BF)
    t = torch.arange(300, device="cuda")
    want, (wloss, wlse) = m.layer_norm(keep, w, w)[0], m.vocab_loss(X, W, t)
    x, Xs = torch.zeros_like(keep), torch.zeros_like(X)
    y, loss, lse = torch.empty_like(x), torch.empty_like(wloss), torch.empty_like(wlse)
    ws = torch.empty(m.flash_mca_vocab_loss_workspace_bytes(300, 900, 64), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    on = side if kind.startswith("side") else torch.cuda.default_stream()
    stream = {"0": 0, "1": 1, "default": on, "side handle": side.cuda_stream, "side": side}[kind]
    torch.cuda.synchronize()
    with torch.cuda.stream(on):
        torch.cuda._sleep(20_000_000)
        x.copy_(keep)
        Xs.copy_(X)
    if explicit:
        m.flash_mca_layer_norm(x, None, w, w, None, y, None, None, stream=stream)
        m.flash_mca_vocab_loss(Xs, W, t, loss, lse, ws, stream=stream)
    else:
        y = m.layer_norm(x, w, w, stream=stream)[0]
        loss, lse = m.vocab_loss(Xs, W, t, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(loss, wloss) and torch.equal(lse, wlse)
