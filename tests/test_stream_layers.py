"""The streaming layers' handling of streams, gradients and the build, without a GPU."""
import contextlib

import pytest
import torch

import block_sparse_attention_hilbert_b200 as svsa
from block_sparse_attention_hilbert_b200 import stream as layers


class _Stream:
    """Stands in for torch.cuda.Stream (and, called, for torch.cuda.stream)."""
    current = None

    def __init__(self, name):
        self.name, self.cuda_stream = name, 0


@pytest.fixture
def streams(monkeypatch):
    """Two fake streams; every allocation, copy and launch of the layers is logged with the stream that was current (or,
    for a launch, the one it was given)."""
    log = []

    @contextlib.contextmanager
    def on(s):
        before, _Stream.current = _Stream.current, s
        try:
            yield
        finally:
            _Stream.current = before

    def note(what, real=None):
        def call(*args, **kw):
            given = kw.get("stream", next((a for a in args if isinstance(a, _Stream)), None))
            log.append((what, _Stream.current, given))
            return real(*args, **kw) if real else None
        return call

    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream.current)
    for name in ("svsa_cache_append", "svsa_cache_attn", "svsa_cache_select", "svsa_qk_norm_rope", "svsa_qk_norm_rope_bwd"):
        monkeypatch.setattr(layers, name, note(name))
    monkeypatch.setattr(torch, "empty", note("empty", torch.empty))
    monkeypatch.setattr(torch.Tensor, "copy_", note("copy_", torch.Tensor.copy_))
    monkeypatch.setattr(torch.Tensor, "zero_", note("zero_", torch.Tensor.zero_))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.append(("record", s, None)))
    return [_Stream("a"), _Stream("b")], log


def _calls():
    B, h, d = 2, 1, 64
    cache = svsa.BlockCache(B, h, d, 200, code="i8", device="cpu")
    rope = svsa.NormRope(d, device="cpu")
    x = torch.zeros(B, h, 3, d, dtype=torch.bfloat16)
    idx, cnt = torch.zeros(B, 3, h, 2, dtype=torch.int32), torch.zeros(B, 3, h, dtype=torch.int32)
    return {"append": lambda s: cache.append(x, x, stream=s), "reset": lambda s: cache.reset(stream=s),
            "select": lambda s: cache.select(x, 2, stream=s), "attend": lambda s: cache.attend(x, stream=s),
            "attend lists": lambda s: cache.attend(x, idx, cnt, stream=s), "norm": lambda s: rope(x, x, stream=s),
            "gradients": lambda s: rope.backward(x, x, x, x, stream=s)}


@pytest.mark.parametrize("name", ["append", "reset", "select", "attend", "attend lists", "norm", "gradients"])
def test_a_call_on_a_stream_does_all_its_work_there(streams, name):
    """A workspace taken from the current stream's memory would go to that stream's next request, or to a call on a third
    stream, while the kernels on the given one still use it."""
    (a, b), log = streams
    call = _calls()[name]
    del log[:]
    for s in (a, b):
        call(s)
        assert log and _Stream.current is None
        work = [e for e in log if e[0] != "record"]
        # on s: current when it happens, and no other stream named
        assert all(now is s and given in (None, s) for _, now, given in work), work
        del log[:]
    call(None)
    assert log and all(now is None and given is None for _, now, given in log)
