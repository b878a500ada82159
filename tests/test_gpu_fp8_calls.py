"""The 8-bit paged cache on the GPU: calls as a server makes them."""
import pytest
import torch

from tests.test_gpu_fp8 import D, Setup, cu_of, i32, tq  # noqa: F401

pytestmark = pytest.mark.gpu


def test_captured_calls_clear_only_what_has_to_be_zero(tq, monkeypatch):  # noqa: F811
    """The workspaces of captured calls, filled with NaN between the replays: the results are the eager calls', and the
    partials that a call does not use are still NaN, so no replay cleared them."""
    gen = torch.Generator().manual_seed(71)
    lens, chunk = [1500, 700], [40, 9]
    s = Setup(tq, gen, lens, 2, 16)
    s.fill(lens)
    q = torch.randn(49, 16, D, generator=gen).bfloat16().cuda()
    cu, start = i32(cu_of(chunk)), i32([n - c for n, c in zip(lens, chunk)])
    ln = i32(lens)
    run = lambda: (s.cache.decode(q[:2], s.table, ln), s.cache.prefill(q, cu, start, s.table))  # noqa: E731
    want = run()
    held = []
    of = tq.Fp8Cache._workspace

    def keep(*args):
        held.append(of(*args))
        return held[-1]
    monkeypatch.setattr(tq.Fp8Cache, "_workspace", keep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    assert len(held) == 2
    for _ in range(3):
        for ws in held:
            ws.fill_(0xFF)
        for x in got:
            x.fill_(7)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for ws in held:
            assert (ws == 0xFF).float().mean() > 0.1
