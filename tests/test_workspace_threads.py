"""Default workspaces of calls made from several host threads."""
import threading
import types

import pytest
import torch

import conv2d_bias_activation_amd as c2d


def _in_thread(call):
    """The value of call() in a thread of its own."""
    got = []
    t = threading.Thread(target=lambda: got.append(call()))
    t.start()
    t.join()
    return got[0]


def test_threads_on_one_stream_have_their_own_buffers(monkeypatch):
    """Two calls of several launches each, queued in turn on one stream, may not hand data on through one buffer; a
    buffer that grows in one thread stays in use in another."""
    monkeypatch.setattr(c2d, "_ws_cache", {})
    monkeypatch.setattr(c2d, "DEFAULT_WORKSPACE_BYTES", 1024)
    device, stream = torch.device("cpu", 0), types.SimpleNamespace(cuda_stream=7)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: torch.no_grad())
    take = lambda need: c2d._default_workspace(device, stream, need)  # noqa: E731
    alive = threading.Barrier(2)
    got = {}

    def worker(name):
        first = take(10)
        alive.wait(30)
        grown = take(5000) if name == "a" else take(10)
        alive.wait(30)
        got[name] = (first, grown, take(10))

    threads = [threading.Thread(target=worker, args=(n,)) for n in "ab"]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    mine = take(10)
    buffers = [mine, got["a"][0], got["a"][1], got["b"][0]]
    assert len({b.data_ptr() for b in buffers}) == 4
    assert got["b"][1] is got["b"][0] and got["b"][2] is got["b"][0]
    assert got["a"][2] is got["a"][1] and got["a"][1].numel() == 5000
    assert take(10) is mine
    assert _in_thread(lambda: take(10)) is not mine


@pytest.mark.gpu
def test_scans_from_two_threads_on_one_stream():
    """Split scans that two threads queue on the default stream at the same time give the bits of the same scans one
    by one."""
    g = torch.Generator(device="cuda").manual_seed(3)
    cases = []
    for tokens, d in ((3000, 64), (5000, 128)):
        u, dt = (torch.randn(1, tokens, d, generator=g, device="cuda") for _ in range(2))
        b = torch.randn(1, tokens, 1, 16, generator=g, device="cuda")
        A = -torch.rand(d, 16, generator=g, device="cuda")
        cases.append(lambda u=u, dt=dt, A=A, b=b: c2d.selective_scan(u, dt, A, b, b, softplus=True))
    want = [call() for call in cases]
    torch.cuda.synchronize()
    got = [[], []]
    start = threading.Barrier(2)

    def worker(i):
        start.wait(30)
        for _ in range(100):
            got[i].append(cases[i]())

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 100
        for y in got[i]:
            assert torch.equal(y, want[i])


@pytest.mark.gpu
def test_default_workspace_belongs_to_the_calls_stream():
    """A buffer that is dropped when a larger one takes its place may only be reused behind the calls that still work
    in it: it has to be allocated on their stream, whichever is current."""
    side = torch.cuda.Stream()
    x = torch.randn(2, 20, 20, 512, device="cuda").bfloat16()
    w = torch.randn(128, 3, 3, 512, device="cuda").bfloat16()
    c2d.conv2d_fused(x, w, pad=1, stream=side)
    ws = c2d._ws_cache[(torch.cuda.current_device(), side.cuda_stream)]
    torch.cuda.synchronize()
    here = [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= ws.data_ptr() < s["address"] + s["total_size"]]
    assert here == [side.cuda_stream]
