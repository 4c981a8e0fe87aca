"""What the binding keeps between calls (CPU): a size by its numbers alone, torch's raw-stream
functions whole."""
import sys
import types

import pytest

import block_scaled_precision_bf16tofp4row_amd as mx

torch = pytest.importorskip("torch")


def test_workspace_size_of_a_tensor_that_changes():
    """The sizes may come as anything that has an int: what is kept goes by the number, not by
    the object that held it once."""
    T = torch.tensor(300)
    few = mx.mxfp4_expert_map_workspace(T, 8, 64)
    T.fill_(9000)
    many = mx.mxfp4_expert_map_workspace(T, 8, 64)
    assert few == mx.mxfp4_expert_map_workspace(300, 8, 64)
    assert many == mx.mxfp4_expert_map_workspace(9000, 8, 64) > few
    assert mx.mxfp4_expert_map_workspace(T=9000, k=8, G=64) == many


def test_raw_stream_functions_are_published_whole(monkeypatch):
    """A thread that finds the raw-stream functions finds all of them: looked at after every
    bytecode of the call that sets them, as another thread may."""
    if not hasattr(torch._C, "_cuda_getCurrentRawStream"):
        pytest.skip("this torch has no raw-stream function")
    names = [n for n in vars(mx) if n in ("_raw_stream", "_device")]
    for n in names:
        monkeypatch.setattr(mx, n, None)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=11))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 70 + device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    seen = []

    def trace(frame, event, arg):
        if frame.f_code is not mx._current_stream.__code__:
            return None
        frame.f_trace_opcodes = True
        if event == "opcode":
            sys.settrace(None)
            if mx._raw_stream is not None:
                seen.append(mx._current_stream())
            sys.settrace(trace)
        return trace

    sys.settrace(trace)
    try:
        assert mx._current_stream() == 11         # the call that sets them
    finally:
        sys.settrace(None)
    assert seen and set(seen) == {73}
    assert mx._current_stream() == 73
