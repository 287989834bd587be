"""The streaming layers' handling of streams, gradients and the build, without a GPU."""
import contextlib

import pytest
import torch

import block_sparse_attention_hilbert_b200 as svsa
from block_sparse_attention_hilbert_b200 import stream as layers


class _Stream:
    """Stands in for torch.cuda.Stream (and, called, for torch.cuda.stream)."""
    current = None

    def __init__(self, name, device="cpu"):
        self.name, self.device, self.cuda_stream = name, torch.device(device), 0


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


@pytest.mark.parametrize("name", ["append", "reset", "select", "attend", "norm", "gradients"])
def test_a_stream_of_another_device_is_refused(streams, name):
    _, log = streams
    call = _calls()[name]
    del log[:]
    with pytest.raises(ValueError, match="stream"):
        call(_Stream("c", "cuda:1"))
    assert not log and _Stream.current is None


def test_norm_and_rotation_record_their_gradients(monkeypatch):
    """Outputs of inputs or weights that require gradients have a grad_fn, whose backward is the library's; what cannot
    carry gradients is refused."""
    B, h, N, d = 1, 2, 5, 64
    seen = []

    def bwd(gq, gk, q, k, wq, wk, cos, sin, pos, iperm, dq, dk, dwq, dwk, p, ws, n, stream=None):
        seen.append((gq, gk, p.rows, iperm))
        dq.fill_(2), dwq.fill_(4)
        if k is not None:
            dk.fill_(3), dwk.fill_(5)

    monkeypatch.setattr(layers, "svsa_qk_norm_rope", lambda *a, **kw: None)
    monkeypatch.setattr(layers, "svsa_qk_norm_rope_bwd", bwd)
    w = torch.ones(d, requires_grad=True)
    rope = svsa.NormRope(d, wq=w, device="cpu")
    x = torch.zeros(B, N, 2 * h, d, dtype=torch.bfloat16)
    q, k = x[:, :, :h].transpose(1, 2), x[:, :, h:].transpose(1, 2)
    yq, yk = rope(q, k)                                    # the weight alone requires gradients
    (yq.float().sum() + 2 * yk.float().sum()).backward()
    assert torch.all(w.grad == 4) and torch.all(seen[0][0] == 1) and torch.all(seen[0][1] == 2)
    assert seen[0][0].is_contiguous() and seen[0][1].is_contiguous()
    x.requires_grad_()
    perm = torch.tensor([4, 3, 2, 1, 0, -1], dtype=torch.int32)
    iperm = torch.tensor([4, 3, 2, 1, 0], dtype=torch.int32)
    q, k = x[:, :, :h].transpose(1, 2), x[:, :, h:].transpose(1, 2)
    yq, yk = rope(q, k, perm=perm, iperm=iperm)
    assert yq.shape == yk.shape == (B, h, 6, d)
    yk.float().sum().backward()                            # (nothing comes back to yq: zeros)
    assert torch.all(x.grad[:, :, :h] == 2) and torch.all(x.grad[:, :, h:] == 3)
    assert torch.all(seen[1][0] == 0) and seen[1][2] == 6 and torch.equal(seen[1][3], iperm)
    y, none = rope(q, None)
    assert none is None
    y.float().sum().backward()
    assert torch.all(x.grad[:, :, :h] == 4)
    with pytest.raises(ValueError):
        rope(q, k, perm=perm)
    out = (torch.empty(B, h, N, d, dtype=torch.bfloat16), torch.empty(B, h, N, d, dtype=torch.bfloat16))
    with pytest.raises(RuntimeError):
        rope(q, k, out=out)
    with torch.no_grad():
        assert rope(q, k, out=out)[0] is out[0] and not rope(q, k)[0].requires_grad


def test_the_library_is_built_without_the_python_module(tmp_path, monkeypatch):
    """Where the Python module does not compile (no Python.h), the C library is linked first and the failure is raised."""
    import ctypes
    import shutil
    import subprocess

    from block_sparse_attention_hilbert_b200 import build
    try:
        build._nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    src, obj = tmp_path / "one.c", tmp_path / "one.o"
    src.write_text("int svsa_one(void) { return 1; }\n")
    subprocess.run(["gcc", "-fPIC", "-c", str(src), "-o", str(obj)], check=True)

    def no_headers(force):
        raise RuntimeError("Python.h: no such file")

    for name, value in (("BUILD", str(tmp_path)), ("LIBDIR", str(tmp_path)), ("LIB", str(tmp_path / "libsvsa.so")),
                        ("BINDING", str(tmp_path / "_svsa_binding.so")), ("_compile", lambda *a: (str(obj), "")),
                        ("_compile_binding", no_headers)):
        monkeypatch.setattr(build, name, value)
    monkeypatch.setattr(build.glob, "glob", lambda pattern: ["one.cu"])
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build()
    assert ctypes.CDLL(str(tmp_path / "libsvsa.so")).svsa_one() == 1
