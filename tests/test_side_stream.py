"""Calls that are given a stream other than the current one and make their outputs themselves: such an output belongs to
the given stream (its memory may otherwise still be in use by the current one, and a fill on the current one may land
behind the call's kernel), and is kept for the current one's reads."""
import contextlib

import pytest
import torch

DEV = torch.device("cuda")


class _Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


class _Tensor:
    """What a call needs of a tensor, and the streams that it was made and recorded on."""

    def __init__(self, made):
        self.made, self.recorded = made, []

    def record_stream(self, s):
        self.recorded.append(s.cuda_stream)


@pytest.mark.parametrize("given", ["other", "current", None])
def test_read_fills_its_outputs_on_the_call_s_stream(monkeypatch, given):
    import bit_kv_cache_ott_gb300 as pkg
    now, other = _Stream(1), _Stream(2)
    state, calls = [now], []

    @contextlib.contextmanager
    def stream(s):
        state.append(s)
        yield
        state.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state[-1])
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: _Tensor(state[-1].cuda_stream))
    c = object.__new__(pkg.ByteCache)
    c.B, c.Hkv, c.d, c._dev, c._h = 1, 1, 64, 0, None
    c._L = type("L", (), {"ott_byte_read": None})
    c._ptr = lambda t, *a: t
    c._call = lambda *a, stream: calls.append(stream)
    s = {"other": other, "current": now, None: None}[given]
    out = c.read(0, 3, stream=s)
    assert calls == [s]
    for t in out:
        assert t.made == (2 if given == "other" else 1)
        assert t.recorded == ([1] if given == "other" else [])


def _calls(ott):
    """(name, a call that takes a stream, its output's shape) of every call that makes an output."""
    B, Hq, Hkv, d, T, n = 2, 4, 2, 128, 300, 3
    g = torch.Generator().manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=g).half().to(DEV)
    K, V, q, k, v = new(B, Hkv, T, d), new(B, Hkv, T, d), new(B, Hq, n, d), new(B, Hkv, n, d), new(B, Hkv, n, d)
    q1 = q[:, :, 0].contiguous()
    pos = torch.arange(B * n, dtype=torch.int32, device=DEV).view(1, B, n)
    byte, two = ott.ByteCache(B, Hq, Hkv, d, 64, max_tokens=T), ott.OTTCache(B, Hq, Hkv, d, max_tokens=T)
    for c in (byte, two):
        c.prefill(K, V)
    return [
        ("byte read", lambda s: byte.read(17, 200, stream=s)[0], (B, Hkv, 200, d)),
        ("byte read past the end", lambda s: byte.read(250, 100, stream=s)[1], (B, Hkv, 100, d)),
        ("byte decode", lambda s: byte.decode_attn(q1, stream=s), (B, Hq, d)),
        ("byte chunk", lambda s: byte.chunk_attn_topk(q, k, v, 2, stream=s), (B, Hq, n, d)),
        ("decode", lambda s: two.decode_attn(q1, stream=s), (B, Hq, d)),
        ("decode, blocks selected", lambda s: two.decode_attn_topk(q1, 1, stream=s), (B, Hq, d)),
        ("decode, window", lambda s: two.decode_attn_window(q1, 50, stream=s), (B, Hq, d)),
        ("chunk", lambda s: two.chunk_attn(q, k, v, stream=s), (B, Hq, n, d)),
        ("rope", lambda s: ott.rope(q, k, pos, (64,), stream=s)[0], (B, Hq, n, d)),
    ], (byte, two)


@pytest.mark.gpu
def test_outputs_of_a_side_stream(ott):
    calls, caches = _calls(ott)
    side = torch.cuda.Stream()
    for name, call, shape in calls:
        want = call(None)
        torch.cuda.synchronize()
        # a block that the current stream has freed and will still read, behind some milliseconds of waiting
        a = torch.ones(shape, dtype=torch.float16, device=DEV)
        at = a.data_ptr()
        torch.cuda._sleep(20_000_000)
        b = a.clone()
        del a
        out = call(side)
        assert out.data_ptr() != at, name
        side.synchronize()
        torch.cuda.synchronize()
        assert (b == 1).all(), name
        assert torch.equal(out, want), name
        # read by the current stream, freed by the caller before that, and the call made again
        torch.cuda.current_stream().wait_stream(side)
        at = out.data_ptr()
        torch.cuda._sleep(20_000_000)
        b = out.clone()
        del out
        again = call(side)
        assert again.data_ptr() != at, name
        torch.cuda.synchronize()
        assert torch.equal(b, want) and torch.equal(again, want), name
        del b, again
    for c in caches:
        c.check_device()
        c.close()


@pytest.mark.gpu
def test_a_side_stream_captured(ott):
    """The capturing stream given by name: outputs come from the graph's own memory."""
    calls, caches = _calls(ott)
    for name, call, _ in calls:
        want = call(None)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            out = call(side)
        out.zero_()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), name
    for c in caches:
        c.check_device()
        c.close()


@pytest.mark.gpu
def test_a_side_stream_of_a_capture(ott):
    """A branch of a graph: the side stream forks from the capturing one and joins it."""
    calls, caches = _calls(ott)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    for name, call, _ in calls:
        want = call(None)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            side.wait_stream(main)
            out = call(side)
            main.wait_stream(side)
            twice = out + out
        out.zero_()
        twice.zero_()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(twice, want + want), name
        del out, twice, graph
    for c in caches:
        c.check_device()
        c.close()
