"""Where the binding's own memory is made: on the stream of the call that uses it."""
import contextlib

import pytest
import torch

from group_affine_bit_gb300 import api


class Streams:
    """torch's stream context, watched; memory is the host's."""

    def __init__(self, monkeypatch):
        self.now, self.made, self.capture = "current", [], 0
        zeros = torch.zeros

        def make(n, **kw):
            t = zeros(n, **{**kw, "device": "cpu"})
            self.made.append((n, self.now))
            return t

        @contextlib.contextmanager
        def stream(s):
            before, self.now = self.now, s
            yield
            self.now = before

        monkeypatch.setattr(torch, "zeros", make)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: f"stream {ptr}")
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capture != 0)
        monkeypatch.setattr(api, "_capture_id", lambda ptr: self.capture)


class Side:
    cuda_stream = 7


def test_a_workspace_is_made_on_the_calls_stream(monkeypatch):
    at = Streams(monkeypatch)
    ws = api.Workspace("cpu")
    ws.get(100, Side())
    ws.get(1000, Side())
    ws.get(50)
    ws.get(5000)
    assert [x for x in at.made if x[0]] == [(100, "stream 7"), (1000, "stream 7"), (5000, "current")]


def test_outgrown_buffers_stay(monkeypatch):
    """A captured graph has their addresses."""
    Streams(monkeypatch)
    ws = api.Workspace("cpu")
    bufs = [ws.get(n) for n in (100, 101, 500)]
    addresses = [b.data_ptr() for b in bufs]
    assert len(set(addresses)) == 3 and [b.data_ptr() for b in ws._kept] == addresses[:2]
    assert sum(b.numel() for b in ws._kept) <= ws.buf.numel()


def test_a_buffer_that_only_a_replay_fills_serves_its_capture_alone(monkeypatch):
    at = Streams(monkeypatch)
    ws = api.Workspace("cpu")
    at.capture = 11
    first = ws.get(100, Side())
    assert ws.get(100, Side()) is first and ws.get(60, Side()) is first
    at.capture = 12
    second = ws.get(100, Side())
    assert second is not first
    at.capture = 0
    third = ws.get(100, Side())
    assert third is not second
    at.capture = 13                # filled before the capture: the capture may use it
    assert ws.get(100, Side()) is third


def problem():
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(700, 16, 2, 128, generator=g).bfloat16().cuda() for _ in "kv")
    table = torch.arange(700, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([11000], dtype=torch.int32, device="cuda")
    qs = [torch.randn(1, n, 4, 128, generator=g).bfloat16().cuda() for n in (1, 32)]
    return api.KVCache(k, v), table, lens, qs


def dirty(nbytes):
    """The allocator's free memory of the current stream, and of a graph's, holds ones."""
    for _ in range(3):
        torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.gpu
def test_a_side_stream_does_not_wait_for_the_current_ones_fill():
    """The current stream is busy and its free memory is not zero: a call on another stream, and one that needs more
    workspace, find theirs filled; an output made for them is not memory that pending work still uses."""
    cache, table, lens, qs = problem()
    want = [api.paged_attention(q, cache, table, lens) for q in qs]
    need = [api.paged_attention_workspace_bytes(cache, q.shape[1], 4) for q in qs]
    assert need[1] > need[0]
    for n in need:
        dirty(n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = api.Workspace()
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(40):
        a = torch.mm(a, a).clamp_(-1, 1)
    got = [api.paged_attention(q, cache, table, lens, workspace=ws, stream=side) for q in qs]
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert int(ws.buf[: api.WORKSPACE_ZEROED].count_nonzero()) == 0
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_a_graph_keeps_a_workspace_that_is_outgrown():
    cache, table, lens, qs = problem()
    want = [api.paged_attention(q, cache, table, lens) for q in qs]
    ws, out = api.Workspace(), torch.empty_like(qs[0])
    api.paged_attention(qs[0], cache, table, lens, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_attention(qs[0], cache, table, lens, out=out, workspace=ws)
    held = ws.buf.numel()
    assert torch.equal(api.paged_attention(qs[1], cache, table, lens, workspace=ws), want[1]) and ws.buf.numel() > held
    dirty(held)
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])


@pytest.mark.gpu
def test_captures_without_a_call_before():
    """Two graphs and a plain call that meet a workspace first during the first capture; the second graph is replayed first."""
    cache, table, lens, qs = problem()
    want = api.paged_attention(qs[0], cache, table, lens)
    dirty(64 << 20)
    ws = api.Workspace()
    graphs, outs = [], []
    for _ in range(2):
        outs.append(torch.empty_like(qs[0]))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(2):
                api.paged_attention(qs[0], cache, table, lens, out=outs[-1], workspace=ws)
    assert torch.equal(api.paged_attention(qs[0], cache, table, lens, workspace=ws), want)
    for i in (1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want)
