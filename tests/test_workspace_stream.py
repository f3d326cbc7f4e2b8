"""A decode without a workspace on a stream of its own: the workspace is made
and zero-filled on that stream, so the call finds it ready and its memory is not
handed out elsewhere while the call runs.  Here with stand-ins for the library
and the streams, on the CPU; on the GPU in test_workspace_stream_gpu.py."""
import contextlib
import types

import pytest
import torch


@pytest.fixture
def recorded(monkeypatch):
    """The binding on CPU tensors: which stream was current at each allocation and each call."""
    from paged_kv_attention_36_b200 import binding
    current, log = ["default"], []

    @contextlib.contextmanager
    def stream(s):
        if s is not None:
            current.append(s)
        yield
        if s is not None:
            current.pop()

    zeros = torch.zeros

    def watched(*size, **kw):
        log.append(("zeros", current[-1]))
        return zeros(*size, **kw)

    class Lib:
        def __getattr__(self, name):
            def fn(*args):
                log.append(("call", name))
                return 0
            return fn

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "zeros", watched)
    monkeypatch.setattr(binding, "lib", Lib())
    monkeypatch.setattr(binding, "_need", lambda *a, **k: None)
    monkeypatch.setattr(binding, "_same_device", lambda *a: None)
    monkeypatch.setattr(binding, "_stream", lambda s: None)
    monkeypatch.setattr(binding, "pa_decode_workspace_bytes", lambda *a: 64)
    monkeypatch.setattr(binding, "pa_decode_shared_prefix_workspace_bytes", lambda *a: 64)
    return binding, log


def _calls(pa):
    q = torch.empty((2, 4, 64), dtype=torch.bfloat16)
    kc = torch.empty((3, 2, 16, 64), dtype=torch.bfloat16)
    k8, v8 = torch.empty((3, 2, 16, 64), dtype=torch.int8), torch.empty((3, 2, 64, 16), dtype=torch.int8)
    kf, vf = k8.view(torch.uint8), v8.view(torch.uint8)
    head, block = torch.ones(2), torch.ones((3, 2))
    bt, cl = torch.ones((2, 1), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    rows, out = torch.empty((2, 2, 64), dtype=torch.bfloat16), torch.empty_like(q)
    return {
        "pa_decode": lambda **k: pa.pa_decode(q, kc, kc, bt, cl, 0.1, out, **k),
        "pa_append_decode": lambda **k: pa.pa_append_decode(rows, rows, cl, q, kc, kc, bt, cl, 0.1, out, **k),
        "pa_decode_shared_prefix": lambda **k: pa.pa_decode_shared_prefix(
            q, kc, kc, bt, cl, 0.1, torch.ones(2, dtype=torch.int32), torch.ones(1, dtype=torch.int32), 2, out, **k),
        "pa_decode_fp8": lambda **k: pa.pa_decode_fp8(q, kf, vf, head, head, bt, cl, 0.1, out, **k),
        "pa_append_decode_fp8": lambda **k: pa.pa_append_decode_fp8(rows, rows, cl, q, kf, vf, head, head, bt, cl, 0.1,
                                                                    out, **k),
        "pa_decode_window": lambda **k: pa.pa_decode_window(q, kc, kc, bt, cl, 0.1, out, window=4, **k),
        "pa_decode_i8": lambda **k: pa.pa_decode_i8(q, k8, v8, block, block, bt, cl, 0.1, out, **k),
    }


@pytest.mark.parametrize("what", ["pa_decode", "pa_append_decode", "pa_decode_shared_prefix", "pa_decode_fp8",
                                  "pa_append_decode_fp8", "pa_decode_window", "pa_decode_i8"])
def test_workspace_is_made_on_the_calls_stream(recorded, what):
    pa, log = recorded
    call = _calls(pa)[what]
    side = types.SimpleNamespace(cuda_stream=0)
    log.clear()
    call(stream=side)
    assert log == [("zeros", side), ("call", what)]
    log.clear()
    call()
    assert log == [("zeros", "default"), ("call", what)]
    log.clear()
    call(stream=side, workspace=torch.empty(64, dtype=torch.uint8))
    assert log == [("call", what)]
